"""The operators around an attention layer with 8-bit operands: block-scaled
FP8 product, per-head RMS norm with RoPE, the FP8 key/value cache and attention
over it; and the products beside it whose weights depend on the token: routing,
experts, low-rank adapters. Re-exported by the package; csrc/binding.cpp checks and marshals the
arguments of the C calls. Nothing here has a backward pass; routing, the experts' weighted sum and
the adapters refuse operands that require a gradient while gradients are recorded."""
import typing

import torch

from . import _check, _lib

__all__ = [
    "fp8_gemm_1x128_128x128", "fp8_gemm_workspace_bytes", "debug_fp8_gemm_kernel", "qk_norm_rope", "Fp8KvCache", "fp8_kv_cache", "kv_cache_append_fp8", "kv_cache_read_fp8",
    "attention_fp8_kv", "attention_fp8_kv_workspace_bytes", "attention_fp8_kv_workspace",
    "RowGroups", "moe_route", "group_rows", "group_rows_workspace_bytes", "fp8_grouped_gemm_1x128_128x128", "fp8_grouped_swiglu_1x128",
    "moe_combine", "lora_add", "lora_add_workspace_bytes",
]


class _NoBinding:
    """Stands for _binding.so where that does not load: the rest of the package
    needs the C library alone."""

    def __init__(self, why):
        self.why = why

    def __getattr__(self, name):
        raise ImportError("the attention layer's operators need fp4_quantized_prep_amd/_binding.so, which is missing or does not "
                          f"load ({self.why}): build it with `python fp4_quantized_prep_amd/build.py`")


try:
    from . import _binding
except ImportError as e:
    _binding = _NoBinding(str(e))
else:
    _binding.set_error(_check)


def _on(stream, tensor, fn, *args):
    """fn(*args) with ``stream`` current: outputs are then allocated from its
    pool and the launch goes to it."""
    if stream.device != tensor.device:
        raise ValueError(f"stream must be on {tensor.device}, got {stream.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


def fp8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of the workspace that :func:`fp8_gemm_1x128_128x128` can use (0: none)."""
    return int(_lib.fp8_gemm_workspace_bytes(M, N, K))


def debug_fp8_gemm_kernel(M: int, N: int, K: int, workspace: bool = True) -> str:
    """Name of the kernel that :func:`fp8_gemm_1x128_128x128` takes for these
    sizes ("" where it refuses them), for tests that mean to reach each."""
    return _lib.iqp_debug_fp8_gemm_kernel(M, N, K, int(workspace)).decode()


def fp8_gemm_1x128_128x128(a, a_scales, w, w_scales, out=None, workspace=None, stream=None):
    """Block-scaled FP8 product ``out = a w^T`` in bf16.

    a: E4M3 [M, K] (uint8 or float8_e4m3fn) and a_scales: the packed words from
    :func:`fp8_quant_1x128_ue8m0` (either layout); w: E4M3 [N, K], any N, and
    w_scales: uint8 [ceil(N/128), K/128] as :func:`fp8_quant_weight_128x128_ue8m0`
    gives them. Rows contiguous, row strides any multiples of 16 up to 2^22.
    workspace: a uint8 tensor of :func:`fp8_gemm_workspace_bytes` bytes for
    products that are split over K (allocated here when None); calls that share
    one must not overlap. Returns ``out``, bf16 [M, N] (rows contiguous where
    passed in).
    """
    args = (a, a_scales, w, w_scales, out, workspace)
    return _binding.fp8_gemm(*args) if stream is None else _on(stream, a, _binding.fp8_gemm, *args)


def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps: float = 1e-6, head_dim: int = 128,
                 rope_layout: str = "half_split", q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head, times the weights, then RoPE on
    each head's first ``cos_sin.shape[1]`` dims, in one pass.

    q, k: bf16 [M, H * head_dim] or [M, H, head_dim], rows contiguous, any row
    strides that are multiples of 8 (column ranges of a fused projection's rows); q_weight,
    k_weight: bf16 [head_dim], finite; positions: int64 [M]; cos_sin: float32 [max_pos,
    rope_dim], the table of :func:`rope_cos_sin_table`, rope_dim a multiple of
    16 up to head_dim. rope_layout: pairs (i, i + rope_dim/2) "half_split", or
    (2i, 2i+1) "interleaved". head_dim: 64, 128 or 256. Returns ``(q_out,
    k_out)`` in the inputs' shapes; they may be q and k themselves.
    """
    args = (q, k, q_weight, k_weight, positions, cos_sin, eps, head_dim, rope_layout, q_out, k_out)
    return _binding.norm_rope(*args) if stream is None else _on(stream, q, _binding.norm_rope, *args)


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


def kv_cache_append_fp8(k, v, cache, block_table, seq_lens, cu_rows, stream=None):
    """Quantises new keys and values into the cache, in place.

    k, v: bf16 [T, n_kv_heads, head_dim] (or flattened rows, any row strides that are
    multiples of 8); rows ``cu_rows[s] .. cu_rows[s+1]`` are the last tokens of
    sequence s, whose length with them is ``seq_lens[s]``. block_table: int32
    [S, max_blocks], the block that holds each ``block_size`` positions. Where a
    block is begun earlier its exponent may grow, and its earlier codes are then
    rounded again. No block may be written through two table entries in one call.
    Returns the cache.
    """
    args = (k, v, *cache, block_table, seq_lens, cu_rows)
    _binding.kv_append(*args) if stream is None else _on(stream, k, _binding.kv_append, *args)
    return cache


def kv_cache_read_fp8(cache, block_table, seq_lens, cu_rows, rows: int, k_out=None, v_out=None, stream=None):
    """Reads keys and values back as bf16: row ``cu_rows[s] + i`` of ``rows`` is
    position ``seq_lens[s] - (cu_rows[s+1] - cu_rows[s]) + i`` of sequence s
    (whole sequences: cu_rows the running sum of seq_lens). Rows that no held
    token belongs to are left as they were in ``k_out`` and ``v_out``; in tensors
    allocated here they hold no particular values. Returns ``(k, v)``, [rows,
    n_kv_heads, head_dim].
    """
    args = (*cache, block_table, seq_lens, cu_rows, rows, k_out, v_out)
    return _binding.kv_read(*args) if stream is None else _on(stream, cache[0], _binding.kv_read, *args)


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
    sees nothing gives zeros. Rows that belong to no sequence (before ``cu_rows[0]``,
    behind ``cu_rows[S]``) are left as they were in ``out``; in a tensor allocated
    here they hold no particular values. ``out`` must not overlap q.
    scale: 1 / sqrt(head_dim) by default, else 2^-64 to 2^64. workspace: a tensor from
    :func:`attention_fp8_kv_workspace` (allocated here when None); calls that
    share one must not overlap. Returns ``out`` in q's shape.
    """
    args = (q, *cache, block_table, seq_lens, cu_rows, scale, window, out, workspace)
    return _binding.attention(*args) if stream is None else _on(stream, q, _binding.attention, *args)


class RowGroups(typing.NamedTuple):
    """A batch's entries sorted by group (expert, adapter), as :func:`group_rows`
    gives them. int32, contiguous."""
    offsets: torch.Tensor  #: [n_groups + 1]: group g has the places offsets[g] .. offsets[g+1] - 1
    rows: torch.Tensor     #: [R]: the (flat) entry at every place, -1 behind the last group
    slots: torch.Tensor    #: in the index's shape: every entry's place, -1 for one in no group


_SCORING = {"softmax": 0, "sigmoid": 1, "sqrt_softplus": 2}


def moe_route(logits, top_k: int, bias=None, scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
              weights=None, experts=None, stream=None):
    """The ``top_k`` experts of every token and their weights.

    logits: float32 or bf16 [M, E], rows contiguous, E up to 1024, top_k up to 64; bias: None or
    float32 [E], added to the scores for the choice alone. scoring: "softmax",
    "sigmoid" or "sqrt_softplus" (sqrt(log(1 + e^z))). The experts are those of the
    largest logits, or with a bias of the largest score plus bias, the lower index
    first where these are equal; a weight is ``scale`` times the score, divided by
    the chosen ones' sum where ``renormalize``. An expert whose logit is -inf comes
    last, with weight 0. Returns ``(weights, experts)``, float32 and int32 [M, top_k].
    """
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {', '.join(_SCORING)}, got {scoring!r}")
    args = (logits, top_k, bias, _SCORING[scoring], renormalize, scale, weights, experts)
    return _binding.route(*args) if stream is None else _on(stream, logits, _binding.route, *args)


def group_rows_workspace_bytes(rows: int, n_groups: int) -> int:
    """Bytes of the workspace that :func:`group_rows` needs for an index of ``rows``
    entries (0: none)."""
    return int(_lib.group_rows_workspace_bytes(rows, n_groups))


def group_rows(index, n_groups: int, out=None, workspace=None, stream=None):
    """Sorts a batch's entries by group, those of a group in their own order.

    index: int32 [M] or [M, k], contiguous: the group of every entry
    (:func:`moe_route`'s experts, or a token's adapter); one outside [0, n_groups)
    is in none. n_groups: up to 1024. out: a :class:`RowGroups` to write to.
    workspace: a uint8 tensor of :func:`group_rows_workspace_bytes` bytes (allocated
    here when None); calls that share one must not overlap. Returns the
    :class:`RowGroups`.
    """
    args = (index, n_groups, *(out or (None, None, None)), workspace)
    return RowGroups(*(_binding.group(*args) if stream is None else _on(stream, index, _binding.group, *args)))


def fp8_grouped_gemm_1x128_128x128(a, a_scales, w, w_scales, groups, gather: bool = False, out=None, stream=None):
    """:func:`fp8_gemm_1x128_128x128` with weights of its own for every group of
    rows: ``out[i] = a[src] w[g]^T`` for every place i of group g.

    a, a_scales: as there; a row for every place (src = i), or with ``gather`` a row
    for every token, whose entries the groups hold (src = rows[i] // k). Less than
    2^31 bytes. w: E4M3 [n_groups, N, K], any N, and w_scales: uint8 [n_groups,
    ceil(N/128), K/128], as :func:`fp8_quant_weight_128x128_ue8m0` gives them for
    each group. Returns ``out``, bf16 [R, N], a row a place; places in no group are
    left as they were (in a tensor allocated here they hold no particular values).
    """
    args = (a, a_scales, w, w_scales, *groups, gather, out)
    return _binding.grouped_gemm(*args) if stream is None else _on(stream, a, _binding.grouped_gemm, *args)


def fp8_grouped_swiglu_1x128(a, a_scales, w, w_scales, groups, gather: bool = False, q=None, q_scales=None, stream=None):
    """The first product of a gated expert and what follows it, in one launch:
    ``h = silu(gate) * up`` with ``[gate, up] = a[src] w[g]^T`` in float32,
    quantised in 1x128 blocks.

    Operands as in :func:`fp8_grouped_gemm_1x128_128x128`, with w [n_groups, 2 I, K]:
    I gate rows, then I up rows, I a multiple of 128. Returns ``(q, q_scales)``: E4M3
    codes (uint8) [R, I] and packed words int32 [R, ceil(I/512)], a row a place, the
    operands of the second product. Places in no group as there.
    """
    args = (a, a_scales, w, w_scales, *groups, gather, q, q_scales)
    return _binding.grouped_swiglu(*args) if stream is None else _on(stream, a, _binding.grouped_swiglu, *args)


def moe_combine(y, groups, weights, shared=None, out=None, stream=None):
    """Every token's weighted sum of its experts' rows, ``out[m] = sum_j
    weights[m, j] y[slots[m, j]] (+ shared[m])``, in float32.

    y: bf16 [R, d], a row a place, d a multiple of 8; weights: float32 in the shape
    of the groups' slots; shared: None or bf16 [M, d] (the shared expert's rows, or a
    residual). Entries in no group are left out. Rows contiguous, strides multiples
    of 8. Returns ``out``, bf16 [M, d]; it may be ``shared`` itself.
    """
    args = (y, *groups, weights, shared, out)
    return _binding.combine(*args) if stream is None else _on(stream, y, _binding.combine, *args)


def lora_add_workspace_bytes(M: int, n_adapters: int, rank: int, K: int) -> int:
    """Bytes of the workspace that :func:`lora_add` needs (0 for one of these sizes that it refuses)."""
    return int(_lib.lora_add_workspace_bytes(M, n_adapters, rank, K))


def lora_add(out, x, lora_a, lora_b, groups, scales=None, workspace=None, stream=None):
    """Adds every token's low-rank adapter to the output of the projection that all
    tokens share, in place: ``out[m] += scales[g] * lora_b[g] (lora_a[g] x[m])``.

    out: bf16 [M, N], any N; x: bf16 [M, K], the projection's input, K a multiple of
    8; rows contiguous, x's strides multiples of 8. lora_a: bf16 [n_adapters, rank,
    K] and lora_b: bf16 [n_adapters, N, rank], contiguous and finite, rank a multiple
    of 8 up to 128; scales: None or float32 [n_adapters]. groups: the
    :func:`group_rows` of one adapter a token; tokens in none keep their rows' bits.
    workspace: a uint8 tensor of :func:`lora_add_workspace_bytes` bytes (allocated here
    when None); calls that share one must not overlap. There is no backward pass: where
    gradients are recorded, tensors that require one are refused. Returns ``out``.
    """
    args = (out, x, lora_a, lora_b, *groups, scales, workspace)
    return _binding.lora(*args) if stream is None else _on(stream, x, _binding.lora, *args)
