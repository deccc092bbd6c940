"""Refusals of the cache calls at the edges of what they accept, on the CPU (host memory stands in for device buffers;
every refusal comes before a launch)."""
import ctypes

import pytest
import torch

from test_kvcache_checks import B, D, G, H, M, P, bf16, cache, calls, fa, i32  # noqa: F401 (fa: fixture)


@pytest.fixture
def library(fa):
    """(attention, accumulate) of the library, as functions of what a case changes."""
    from blackwell_nvfp4_quantize_gb300 import kvcache as kv

    L = kv._L()
    buf = ctypes.create_string_buffer(4096)
    at = (ctypes.addressof(buf) + 255) // 256 * 256

    def query_args(k_exp=0, heads=H, rows=B, sequences=B, max_pages=M, cu=None, group=G, max_new=1, scale=0.1, cap=0.0):
        return (kv._Cache(at, P, heads, D, k_exp, 0), kv._Batch(at, at, cu, sequences, max_pages, rows), at, H * G * D, D,
                group, max_new, scale, cap, 0, None)

    def attention(**kw):
        return L.fp4attn_kv_attention(*query_args(**kw), at, at, at, 1 << 40, None), buf

    def accumulate(**kw):
        return L.fp4attn_kv_accumulate(*query_args(**kw), at, at, 1 << 20, 1.0, None), buf

    return lambda **kw: (attention(**kw)[0], accumulate(**kw)[0])


def test_factors_that_fp32_does_not_hold(fa, library):
    bad = (fa.FP4ATTN_ERR_INVALID_ARG,) * 2
    # scores' factor below fp32's normal numbers; caps that would push it there, or overflow
    for kw in (dict(scale=1e-39), dict(k_exp=-32, scale=1e-30), dict(cap=2.0 ** 91), dict(cap=3e38)):
        assert library(**kw) == bad, kw
    for kw in (dict(k_exp=-32, scale=1e-28), dict(cap=2.0 ** 90), dict(cap=2.0 ** 90, scale=1e-30)):
        assert library(rows=0, max_new=0, **kw) == (fa.FP4ATTN_OK,) * 2, kw


def test_work_that_32_bits_do_not_count(fa, library):
    """Units of all tiles, and the runs they are rounded up to, are counted in 32 bits."""
    uns = (fa.FP4ATTN_ERR_UNSUPPORTED,) * 2
    # 337 sequences of 6223 KV heads and 1024 pages: 2^31 - 1024 units
    assert library(sequences=337, rows=337, heads=6223, max_pages=1024, group=1) == uns
    assert library(sequences=1, rows=1, heads=65, max_pages=2 ** 24, group=1) == uns
    assert library(sequences=1, rows=0, max_new=0, heads=63, max_pages=2 ** 24, group=1) == (fa.FP4ATTN_OK,) * 2


def test_workspace_of_sizes_that_the_call_refuses(fa):
    from blackwell_nvfp4_quantize_gb300 import kvcache as kv

    n = ctypes.c_size_t()
    f = kv._L().fp4attn_kv_attention_workspace_bytes
    big = 2 ** 31 - 1
    for heads, seqs, pages, group, new in ((H, 2049, 8, 1, 1), (H, 4, 2 ** 24 + 1, 1, 1), (70000, 4, 8, 1, 1),
                                           (40000, 4, 8, 2, 1), (big, big, big, 1, 64), (H, 4, 8, 1, 2 ** 24 + 1)):
        assert f(heads, 128, seqs, pages, group, new, ctypes.byref(n)) == fa.FP4ATTN_ERR_UNSUPPORTED, (heads, seqs, pages)


@pytest.mark.parametrize("name", ["append", "attention", "accumulate"])
def test_strides_of_a_dimension_of_one_do_not_matter(fa, name):
    """A single row, or a single head, of a wider tensor: what its stride says addresses nothing."""
    f, a = calls(fa)[name]
    rows = [x for x in ("k", "v", "q") if x in a]
    one = dict(cache=cache(fa, pages=torch.zeros((P, 1, 72 * D), dtype=torch.uint8)), table=i32(1, M), lens=i32(1))
    if name == "accumulate":
        one.update(lse=torch.zeros((1, 1)), weights=torch.zeros((1, 1, 64 * M)))
    x = torch.empty_strided((1, 1, D), (D + 3, 2 * D + 1, 1), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):  # the last check: everything else is in order
        f(**{**a, **one, **{n: x for n in rows}})
    x = torch.empty_strided((3, 1, D), (D + 3, D, 1), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiples of 8"):
        f(**{**a, **one, **{n: x for n in rows}, **dict(table=i32(3, M), lens=i32(3)),
             **(dict(lse=torch.zeros((3, 1)), weights=torch.zeros((3, 1, 64 * M))) if name == "accumulate" else {})})


def test_numbers_that_32_bits_do_not_hold(fa):
    """They are refused, not cut to their low bits."""
    for f, a in calls(fa).values():
        for bad in (cache(fa, k_exp=2 ** 40), cache(fa, v_exp=1.5), cache(fa, k_exp=None)):
            with pytest.raises(ValueError, match="32 bits"):
                f(**{**a, "cache": bad})
    f, a = calls(fa)["read"]
    with pytest.raises(ValueError, match="32 bits"):
        f(**{**a, "total": B * 2 ** 32})
    for call in (lambda: fa.kv_page_bytes(2 ** 32 + 1, 64), lambda: fa.kv_page_bytes(1, 2 ** 32 + 64),
                 lambda: fa.kv_attention_workspace_bytes(H, D, 2 ** 32 + 1, M, 1, 1),
                 lambda: fa.kv_attention_workspace_bytes(H, D, 1, M, 1, 2 ** 32 + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
