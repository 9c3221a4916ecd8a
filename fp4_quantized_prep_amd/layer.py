"""The operators around an attention layer with 8-bit operands: block-scaled
FP8 product, per-head RMS norm with RoPE, the FP8 key/value cache and attention
over it. Re-exported by the package; checks and marshals arguments only."""
import typing

import torch

from . import IQP_ROPE_INTERLEAVED, _bytes_u8, _check, _lib, _require

__all__ = [
    "fp8_gemm_1x128_128x128", "qk_norm_rope", "Fp8KvCache", "fp8_kv_cache", "kv_cache_append_fp8", "kv_cache_read_fp8",
    "attention_fp8_kv", "attention_fp8_kv_workspace_bytes", "attention_fp8_kv_workspace",
]


def _run(fn, where: str, dev: torch.device, stream, args):
    """One C call with ``dev`` current (the library launches on the current
    device) and the stream's handle as its last argument."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream must be on {dev}, got {stream.device}")
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream.cuda_stream)
    if st:
        _check(st, where)


def _empty(shape, dtype, dev, stream):
    """An output from the pool of the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _gpu(t, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.device


def fp8_gemm_1x128_128x128(a, a_scales, w, w_scales, out=None, stream=None):
    """Block-scaled FP8 product ``out = a w^T`` in bf16.

    a: E4M3 [M, K] (uint8 or float8_e4m3fn) and a_scales: the packed words from
    :func:`fp8_quant_1x128_ue8m0` (either layout); w: E4M3 [N, K], any N, and
    w_scales: uint8 [ceil(N/128), K/128] as :func:`fp8_quant_weight_128x128_ue8m0`
    gives them. Rows contiguous, any row strides that are multiples of 16.
    Returns ``out``, bf16 [M, N] (rows contiguous where passed in).
    """
    dev = _gpu(a, "a")
    a, w = _bytes_u8(a), _bytes_u8(w)
    _require(a, "a", torch.uint8, dev, 2)
    _require(a_scales, "a_scales", torch.int32, dev, 2)
    _require(w, "w", torch.uint8, dev, 2)
    _require(w_scales, "w_scales", torch.uint8, dev, 2)
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w must be [N, {K}], got {tuple(w.shape)}")
    if tuple(a_scales.shape) != (M, (K // 128 + 3) // 4):
        raise ValueError(f"a_scales must be [{M}, {(K // 128 + 3) // 4}] (one packed word per 512 columns), got "
                         f"{tuple(a_scales.shape)}")
    if tuple(w_scales.shape) != ((N + 127) // 128, K // 128):
        raise ValueError(f"w_scales must be [{(N + 127) // 128}, {K // 128}], got {tuple(w_scales.shape)}")
    if out is None:
        out = _empty((M, N), torch.bfloat16, dev, stream)
    _require(out, "out", torch.bfloat16, dev, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be [{M}, {N}], got {tuple(out.shape)}")
    if M and N and (a.stride(1) != 1 or w.stride(1) != 1 or out.stride(1) != 1 or w_scales.stride(1) != 1):
        raise ValueError("a, w, w_scales and out need contiguous rows")
    _run(_lib.fp8_gemm_1x128_128x128, "fp8_gemm_1x128_128x128", dev, stream,
         (a.data_ptr(), a.stride(0), a_scales.data_ptr(), a_scales.stride(0), a_scales.stride(1), w.data_ptr(),
          w.stride(0), w_scales.data_ptr(), w_scales.stride(0), M, N, K, out.data_ptr(), out.stride(0)))
    return out


def _heads(t, name: str, dev, head_dim: int, heads=None, dtype=torch.bfloat16):
    """Rows of heads, [M, H, D] or [M, H * D], contiguous within a row ->
    (heads, row stride)."""
    if t.dim() == 3:
        ok = t.shape[2] == head_dim and t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == head_dim)
        h = t.shape[1]
    elif t.dim() == 2:
        ok = t.shape[1] % head_dim == 0 and (t.stride(1) == 1)
        h = t.shape[1] // head_dim
    else:
        ok, h = False, 0
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not ok and t.numel() or heads is not None and h != heads:
        raise ValueError(f"{name} must be [rows, heads, {head_dim}] or [rows, heads * {head_dim}] with contiguous rows"
                         f"{'' if heads is None else f' of {heads} heads'}, got shape {tuple(t.shape)}, strides "
                         f"{t.stride()}")
    return h, t.stride(0)


def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps: float = 1e-6, head_dim: int = 128,
                 rope_layout: str = "half_split", q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head, times the weights, then RoPE on
    each head's first ``cos_sin.shape[1]`` dims, in one pass.

    q, k: bf16 [M, H * head_dim] or [M, H, head_dim], rows contiguous, any row
    strides that are multiples of 8 (column ranges of a fused projection's rows); q_weight,
    k_weight: bf16 [head_dim]; positions: int64 [M]; cos_sin: float32 [max_pos,
    rope_dim], the table of :func:`rope_cos_sin_table`, rope_dim a multiple of
    16 up to head_dim. rope_layout: pairs (i, i + rope_dim/2) "half_split", or
    (2i, 2i+1) "interleaved". head_dim: 64, 128 or 256. Returns ``(q_out,
    k_out)`` in the inputs' shapes; they may be q and k themselves.
    """
    dev = _gpu(q, "q")
    if rope_layout not in ("half_split", "interleaved"):
        raise ValueError("rope_layout must be 'half_split' or 'interleaved'")
    M = q.shape[0] if q.dim() else 0
    Hq, ldq = _heads(q, "q", dev, head_dim)
    Hk, ldk = _heads(k, "k", dev, head_dim)
    _require(positions, "positions", torch.int64, dev, 1)
    _require(cos_sin, "cos_sin", torch.float32, dev, 2)
    _require(q_weight, "q_weight", torch.bfloat16, dev, 1)
    _require(k_weight, "k_weight", torch.bfloat16, dev, 1)
    if k.shape[0] != M or positions.shape[0] != M:
        raise ValueError("q, k and positions need one row per token")
    if q_weight.shape[0] != head_dim or k_weight.shape[0] != head_dim:
        raise ValueError(f"q_weight and k_weight need {head_dim} values")
    if not (positions.is_contiguous() and cos_sin.is_contiguous() and q_weight.is_contiguous() and
            k_weight.is_contiguous()):
        raise ValueError("positions, cos_sin and the weights must be contiguous")
    if q_out is None:
        q_out = _empty(q.shape, torch.bfloat16, dev, stream)
    if k_out is None:
        k_out = _empty(k.shape, torch.bfloat16, dev, stream)
    ldqo, ldko = _heads(q_out, "q_out", dev, head_dim, Hq)[1], _heads(k_out, "k_out", dev, head_dim, Hk)[1]
    if q_out.shape[0] != M or k_out.shape[0] != M:
        raise ValueError("q_out and k_out need one row per token")
    max_pos, rope_dim = cos_sin.shape
    _run(_lib.qk_norm_rope, "qk_norm_rope", dev, stream,
         (q.data_ptr(), ldq, k.data_ptr(), ldk, M, Hq, Hk, head_dim, rope_dim, q_weight.data_ptr(), k_weight.data_ptr(),
          eps, positions.data_ptr(), cos_sin.data_ptr(), max_pos, q_out.data_ptr(), ldqo, k_out.data_ptr(), ldko,
          IQP_ROPE_INTERLEAVED if rope_layout == "interleaved" else 0))
    return q_out, k_out


class Fp8KvCache(typing.NamedTuple):
    """The paged FP8 key/value cache of one layer: E4M3 codes and one UE8M0
    byte per block and head, for the keys and for the values (value = code *
    2^(byte - 127)). All contiguous."""
    k: torch.Tensor         #: uint8 [n_blocks, n_kv_heads, block_size, head_dim]
    v: torch.Tensor         #: uint8 [n_blocks, n_kv_heads, head_dim, block_size]
    k_scales: torch.Tensor  #: uint8 [n_blocks, n_kv_heads]
    v_scales: torch.Tensor  #: uint8 [n_blocks, n_kv_heads]


def fp8_kv_cache(n_blocks: int, n_kv_heads: int, head_dim: int = 128, block_size: int = 64, device="cuda"):
    """An empty :class:`Fp8KvCache` (head_dim 64 or 128; block_size 16, 32, 64
    or 128 tokens)."""
    if head_dim not in (64, 128) or block_size not in (16, 32, 64, 128):
        raise ValueError("head_dim must be 64 or 128, block_size 16, 32, 64 or 128")
    z = dict(dtype=torch.uint8, device=device)
    return Fp8KvCache(torch.zeros((n_blocks, n_kv_heads, block_size, head_dim), **z),
                      torch.zeros((n_blocks, n_kv_heads, head_dim, block_size), **z),
                      torch.zeros((n_blocks, n_kv_heads), **z), torch.zeros((n_blocks, n_kv_heads), **z))


def _cache_args(cache, dev):
    """Checks of a cache; (n_blocks, heads, block size, head dim)."""
    k, v, ks, vs = cache
    _require(k, "cache.k", torch.uint8, dev, 4)
    _require(v, "cache.v", torch.uint8, dev, 4)
    _require(ks, "cache.k_scales", torch.uint8, dev, 2)
    _require(vs, "cache.v_scales", torch.uint8, dev, 2)
    n, h, b, d = k.shape
    if tuple(v.shape) != (n, h, d, b) or tuple(ks.shape) != (n, h) or tuple(vs.shape) != (n, h):
        raise ValueError(f"cache.v must be [{n}, {h}, {d}, {b}] and the scales [{n}, {h}]")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    return n, h, b, d


def _batch_args(block_table, seq_lens, cu_rows, dev):
    _require(block_table, "block_table", torch.int32, dev, 2)
    _require(seq_lens, "seq_lens", torch.int32, dev, 1)
    _require(cu_rows, "cu_rows", torch.int32, dev, 1)
    S, width = block_table.shape
    if seq_lens.shape[0] != S or cu_rows.shape[0] != S + 1:
        raise ValueError(f"seq_lens must hold {S} entries and cu_rows {S + 1}")
    if not seq_lens.is_contiguous() or not cu_rows.is_contiguous() or (S and width and block_table.stride(1) != 1):
        raise ValueError("seq_lens and cu_rows must be contiguous, block_table's rows too")
    return block_table.data_ptr(), max(block_table.stride(0), width), width, seq_lens.data_ptr(), cu_rows.data_ptr(), S


def kv_cache_append_fp8(k, v, cache, block_table, seq_lens, cu_rows, stream=None):
    """Quantises new keys and values into the cache, in place.

    k, v: bf16 [T, n_kv_heads, head_dim] (or flattened rows, any row strides that are
    multiples of 8); rows ``cu_rows[s] .. cu_rows[s+1]`` are the last tokens of
    sequence s, whose length with them is ``seq_lens[s]``. block_table: int32
    [S, max_blocks], the block that holds each ``block_size`` positions. Where a
    block is begun earlier its exponent may grow, and its earlier codes are then
    rounded again. A block must not be written for two sequences in one call.
    Returns the cache.
    """
    dev = _gpu(k, "k")
    n, h, b, d = _cache_args(cache, dev)
    ldk, ldv = _heads(k, "k", dev, d, h)[1], _heads(v, "v", dev, d, h)[1]
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v need one row per token")
    table, ldt, width, lens, cu, S = _batch_args(block_table, seq_lens, cu_rows, dev)
    _run(_lib.kv_cache_append_fp8, "kv_cache_append_fp8", dev, stream,
         (k.data_ptr(), ldk, v.data_ptr(), ldv, T, h, d, cache.k.data_ptr(), cache.v.data_ptr(),
          cache.k_scales.data_ptr(), cache.v_scales.data_ptr(), n, b, table, ldt, width, lens, cu, S))
    return cache


def kv_cache_read_fp8(cache, block_table, seq_lens, cu_rows, rows: int, k_out=None, v_out=None, stream=None):
    """Reads keys and values back as bf16: row ``cu_rows[s] + i`` of ``rows`` is
    position ``seq_lens[s] - (cu_rows[s+1] - cu_rows[s]) + i`` of sequence s
    (whole sequences: cu_rows the running sum of seq_lens). Rows that no held
    token belongs to are left as they were. Returns ``(k, v)``, [rows,
    n_kv_heads, head_dim].
    """
    dev = _gpu(cache.k, "cache.k")
    n, h, b, d = _cache_args(cache, dev)
    if k_out is None:
        k_out = _empty((rows, h, d), torch.bfloat16, dev, stream)
    if v_out is None:
        v_out = _empty((rows, h, d), torch.bfloat16, dev, stream)
    ldk, ldv = _heads(k_out, "k_out", dev, d, h)[1], _heads(v_out, "v_out", dev, d, h)[1]
    if k_out.shape[0] != rows or v_out.shape[0] != rows:
        raise ValueError(f"k_out and v_out need {rows} rows")
    table, ldt, width, lens, cu, S = _batch_args(block_table, seq_lens, cu_rows, dev)
    _run(_lib.kv_cache_read_fp8, "kv_cache_read_fp8", dev, stream,
         (cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scales.data_ptr(), cache.v_scales.data_ptr(), n, b, h, d, table,
          ldt, width, lens, cu, S, k_out.data_ptr(), ldk, v_out.data_ptr(), ldv, rows))
    return k_out, v_out


def attention_fp8_kv_workspace_bytes(head_dim: int = 128) -> int:
    """Bytes of the workspace that :func:`attention_fp8_kv` needs."""
    return int(_lib.attention_fp8_kv_workspace_bytes(head_dim))


def attention_fp8_kv_workspace(head_dim: int = 128, device="cuda"):
    """A workspace for :func:`attention_fp8_kv` (its contents do not matter)."""
    return torch.empty(attention_fp8_kv_workspace_bytes(head_dim), dtype=torch.uint8, device=device)


def attention_fp8_kv(q, cache, block_table, seq_lens, cu_rows, scale: float = None, window: int = 0, out=None,
                     workspace=None, stream=None):
    """Causal attention of bf16 queries over the FP8 cache.

    q: bf16 [T, n_heads, head_dim] (or flattened rows, any row strides that are
    multiples of 8), n_heads a multiple of the cache's; rows ``cu_rows[s] ..
    cu_rows[s+1]`` are the last tokens of sequence s, of ``seq_lens[s]`` tokens with
    them, all of which the cache holds (append first). A query at position p
    sees the positions up to p, with ``window`` > 0 only the last ``window`` of
    them; block_table entries outside [0, n_blocks) hold nothing. A query that
    sees nothing gives zeros; rows behind ``cu_rows[S]`` are left as they were.
    scale: 1 / sqrt(head_dim) by default. workspace: a tensor from
    :func:`attention_fp8_kv_workspace` (allocated here when None); calls that
    share one must not overlap. Returns ``out`` in q's shape.
    """
    dev = _gpu(q, "q")
    n, h, b, d = _cache_args(cache, dev)
    Hq, ldq = _heads(q, "q", dev, d)
    if h == 0 or Hq % h:
        raise ValueError(f"q needs a multiple of the cache's {h} heads, got {Hq}")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    ldo = _heads(out, "out", dev, d, Hq)[1]
    if out.shape[0] != q.shape[0]:
        raise ValueError("out needs one row per query")
    if workspace is None:
        workspace = _empty((attention_fp8_kv_workspace_bytes(d),), torch.uint8, dev, stream)
    else:
        _require(workspace, "workspace", torch.uint8, dev, 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    table, ldt, width, lens, cu, S = _batch_args(block_table, seq_lens, cu_rows, dev)
    _run(_lib.attention_fp8_kv, "attention_fp8_kv", dev, stream,
         (q.data_ptr(), ldq, q.shape[0], Hq, h, d, cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scales.data_ptr(),
          cache.v_scales.data_ptr(), n, b, table, ldt, width, lens, cu, S, d ** -0.5 if scale is None else scale, window,
          out.data_ptr(), ldo, workspace.data_ptr(), workspace.numel()))
    return out
