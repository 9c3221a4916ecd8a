"""The operators around an attention layer with 8-bit operands: block-scaled
FP8 product, per-head RMS norm with RoPE, the FP8 key/value cache and attention
over it. Re-exported by the package; csrc/binding.cpp checks and marshals the
arguments of the C calls."""
import typing

import torch

from . import _check, _lib

__all__ = [
    "fp8_gemm_1x128_128x128", "fp8_gemm_workspace_bytes", "debug_fp8_gemm_kernel", "qk_norm_rope", "Fp8KvCache", "fp8_kv_cache", "kv_cache_append_fp8", "kv_cache_read_fp8",
    "attention_fp8_kv", "attention_fp8_kv_workspace_bytes", "attention_fp8_kv_workspace",
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