"""The 4-bit key/value cache on a GPU at the edges of what its calls accept."""
import numpy as np
import pytest
import torch

import _kv_reference as ref
from test_gpu_kvcache import Setup, WIDE, check_attention, fa, ok, rows_alone  # noqa: F401 (fa: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_that_alternate_give_the_same_bits(fa, D):
    """Operands, and whether a page counts, pass between warps and CTAs: what is left of the call before, which had
    other data and other bad pages in the same places, must not show."""
    s = Setup(fa, [700, 200, 1300, 64], [300, 140, 90, 64], H=4, D=D, seed=7)
    s.append_all()
    ok(fa)
    good = s.d_table
    tables = [good, good.clone(), good.clone()]
    tables[1][0, 3], tables[1][2, 8], tables[1][2, 20] = -1, s.P, -1
    tables[2][0, 4], tables[2][1, 0], tables[2][2, 9] = s.P + 1, -1, -1
    qs = [s.queries(3).cuda() for _ in tables]
    want = []
    for turn in range(40):
        i = turn % 3
        s.d_table = tables[i]
        o, lse = rows_alone(fa, s, qs[i])
        if turn < 3:
            want.append((o, lse))
        else:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]), turn
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FP4ATTN_ERR_BAD_INDEX
    s.store_all()
    cu, lens = s.cu, s.lens
    o, lse, to, tl = ref.attention(qs[0].double().cpu().numpy(), s.pool, s.table, lens, cu, D, s.k_exp, s.v_exp, D ** -0.5,
                                   prompt=True)
    assert np.all(np.abs(want[0][0].double().cpu().numpy() - o) <= to)
    assert np.all(np.abs(want[0][1].double().cpu().numpy() - lse) <= tl)
    assert all(torch.all(torch.isfinite(o)) for o, _ in want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,columns", [([1, 3], 0), ([1, 3], WIDE), ([70, 90], 0)])
@pytest.mark.parametrize("k_exp,scale,window", [(-32, 1.0, 0), (-28, 1.0, 40), (32, 1.0, 0), (0, 1e-9, 0), (-10, 1e-6, 40)])
def test_zero_and_tiny_rows_at_every_scale(fa, D, news, columns, k_exp, scale, window):
    """A masked score stays masked where the factor from products to scores leaves fp32's normal numbers."""
    s = Setup(fa, [150, 90], news, D=D, seed=3, k_exp=k_exp, v_exp=k_exp, kv_scale=2.0 ** k_exp, columns=columns)
    q = s.queries(2, 2.0 ** -k_exp)
    q[0], q[2, 1] = 0, 0
    q[1] *= 2.0 ** -80
    q[3, 0] *= 2.0 ** -60
    scale *= D ** -0.5
    kw = dict(window=window) if window else {}
    check_attention(fa, s, 2, q=q, scale=scale, **kw)
    common = dict(cu=s.d_cu, max_new=max(news), softmax_scale=scale, window=window)
    _, lse = fa.kv_attention(q.cuda(), s.cache, s.d_table, s.d_lens, **common)
    w = torch.zeros((s.B, s.H, s.M * 64), device="cuda")
    fa.kv_accumulate(q.cuda(), lse, w, s.cache, s.d_table, s.d_lens, **common)
    ok(fa)
    rw = np.zeros(w.shape)
    tw = ref.attention(q.double().numpy(), s.pool, s.table, s.lens, s.cu, D, k_exp, k_exp, scale, weights=rw,
                       lse_in=lse.double().cpu().numpy(), window=window)[4]
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= tw)


@pytest.mark.parametrize("news", [[1, 3], [70, 90]])
@pytest.mark.parametrize("cap,scale", [(2.0 ** 90, 1.0), (1e20, 1.0), (1e20, 2.0 ** -100)])
def test_caps_far_above_the_scores_change_nothing(fa, news, cap, scale):
    """c tanh(s / c) is s to (s / c)^2 / 3 of itself.  The kernel's tanh adds 2^-21 of each score."""
    s = Setup(fa, [150, 90], news, D=128, seed=3)
    s.append_all()
    s.store_all()
    q = s.queries(2, 1 / scale)
    scale *= 128 ** -0.5
    o, lse = fa.kv_attention(q.cuda(), s.cache, s.d_table, s.d_lens, cu=s.d_cu, max_new=max(news), softmax_scale=scale,
                             softcap=cap)
    ok(fa)
    ro, rl, to, tl = ref.attention(q.double().numpy(), s.pool, s.table, s.lens, s.cu, 128, s.k_exp, s.v_exp, scale,
                                   prompt=max(news) > 3)
    most = max(np.abs(ref.gather(s.pool, s.table, b, s.lens[b], h, 128, s.k_exp, s.v_exp)[0]
                      @ q[s.cu[b]:s.cu[b + 1], 2 * h:2 * h + 2].double().numpy().reshape(-1, 128).T).max() * scale
               for b in range(2) for h in range(s.H))
    ds = 2.0 ** -21 * most
    vmax = float(torch.cat(s.v).abs().max()) * 1.2  # (stored values are off by a sixth at most)
    assert np.all(np.abs(o.double().cpu().numpy() - ro) <= to + 2 * ds * vmax)
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= tl + ds)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,columns", [([3, 2], 0), ([3, 2], WIDE), ([70, 90], 0)])
@pytest.mark.parametrize("window", [1, 20, 64, 130])
def test_pages_before_the_window_may_be_gone(fa, D, news, columns, window):
    """What every query's window has left behind is not looked at: pages may be back in the pool (-1 in the table, or
    in use by others), what shares a page with visible tokens may hold NaN scales."""
    s = Setup(fa, [500, 333], news, D=D, seed=5, columns=columns)
    s.append_all()
    q = s.queries(2).cuda()
    want = rows_alone(fa, s, q, window=window)
    lse0 = want[1].clone()
    w = [torch.zeros((2, s.H, s.M * 64), device="cuda") for _ in range(2)]
    common = dict(cu=s.d_cu, max_new=max(news), window=window)
    fa.kv_accumulate(q, lse0, w[0], s.cache, s.d_table, s.d_lens, **common)
    ok(fa)
    for b, (L, n) in enumerate(zip(s.lens, news)):
        first = L - n - window + 1  # the first slot that some query sees
        for slot in range(first // 64 * 64, first):
            for h in range(s.H):
                for at in ref.offsets(slot % 64, D):
                    s.cache.pages[int(s.table[b, slot // 64]), h, torch.from_numpy(at).cuda()] = 0xFF
        s.d_table[b, :first // 64] = torch.tensor([-1, s.P] * 8, device="cuda")[:first // 64]
    o, lse = rows_alone(fa, s, q, window=window)
    fa.kv_accumulate(q, lse0, w[1], s.cache, s.d_table, s.d_lens, **common)
    ok(fa)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(w[0], w[1])


def stream_calls(fa, s, q, big):
    """Every call that makes its outputs, for a given stream."""
    w = torch.rand((2, s.H, s.M * 64), device="cuda")
    nt = torch.from_numpy(s.spare[:4].reshape(2, 2).copy()).cuda()
    cu = torch.tensor([0, 60, 100], dtype=torch.int32, device="cuda")
    return {
        "read": lambda st: fa.kv_read(s.cache, s.d_table, s.d_lens, 100, cu=cu, stream=st),
        "attention": lambda st: fa.kv_attention(q, s.cache, s.d_table, s.d_lens, stream=st),
        "prompt": lambda st: fa.kv_attention(big, s.cache, s.d_table, s.d_lens, cu=cu, max_new=60, stream=st),
        "evict": lambda st: fa.kv_evict(s.cache, w, s.d_table, s.d_lens, nt, 66, stream=st),
    }


@pytest.mark.parametrize("name", ["read", "attention", "prompt", "evict"])
@pytest.mark.parametrize("columns", [0, WIDE])
@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_on_another_stream(fa, name, columns, handle):
    """Neither do kernels of the current stream that are still to come write to the memory that a call on another
    stream gets, nor does the next such call get memory that the current stream still reads."""
    s = Setup(fa, [700, 190], [1, 1], seed=2, spare=6, columns=columns)
    s.append_all()
    q, big = (Setup._bf16(s.rng.standard_normal((n, 4, s.D))).cuda() for n in (2, 100))
    call = stream_calls(fa, s, q, big)[name]
    want = call(None)
    side = torch.cuda.Stream()
    st = side.cuda_stream if handle else side
    ok(fa)
    sizes = [x.numel() * x.element_size() for x in want] + [1 << 20, 1 << 22, 1 << 24, 1 << 26]
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(400_000_000)
    for x in junk:
        x.fill_(0x7F)  # after the sleep
    del junk, x
    got = call(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # read late on the current stream, while the other one goes on
    torch.cuda._sleep(400_000_000)
    late = [x.clone() for x in got]
    del got
    with torch.cuda.stream(side):
        for _ in range(3):
            for x in call(st):
                x.fill_(3)
    ok(fa)
    assert all(torch.equal(a, b) for a, b in zip(late, want))


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_write_every_row(fa, D):
    """No row of a sequence is left as it was, whatever the batch (the kernel's shared memory grows with it)."""
    for B in (1, 3, 130, 2048):
        news = [70 if b % 700 == 0 else 1 for b in range(B)]
        s = Setup(fa, news, news, H=1, D=D, seed=B)
        s.append_all()
        q = s.queries(1).cuda()
        o = torch.full(q.shape, 1000.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 1000.0, device="cuda")
        rows_alone(fa, s, q, o=o, lse=lse)
        ok(fa)
        assert torch.all(o.abs() < 100) and torch.all(lse.abs() < 100)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news", [2, 40])
def test_a_long_tail_of_light_tokens_counts(fa, D, news):
    """2^21 tokens of 2^-28.5 of the first one's weight: together 2^-7.5 of the result.  A sequence as long as this
    holds P as 2^7 p or more of its maximum, and fp16 is off by half of 2^-24 at most: F = 2^-32 per token in place
    of the 2^-28 of the restatement's bound.  (So many sequences that a problem lies in one or two runs.)"""
    B, G, L = 160, 2, 2 ** 21
    cache = fa.empty_kv_cache(2, 1, D, "cuda", v_exp=0)
    table = torch.ones((B, L // 64), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    k, v = torch.zeros((128, 1, D)), torch.ones((128, 1, D))
    k[0], v[0] = 1.0, 0.0
    one = torch.tensor([128], dtype=torch.int32, device="cuda")
    fa.kv_append(k.bfloat16().cuda(), v.bfloat16().cuda(), cache, table[:1, :2].contiguous(), one)
    k, v = (x[:, 0].double() for x in fa.kv_read(cache, table[:1, :2].contiguous(), one, 128))
    q = torch.ones((B * news, G, D), dtype=torch.bfloat16, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    scale = 28.5 * np.log(2) / float(k[0].sum())
    o, lse = fa.kv_attention(q, cache, table, lens, softmax_scale=scale)
    ok(fa)
    i = torch.arange(news, device="cuda").double().reshape(-1, 1, 1)
    light = 2.0 ** -28.5 * (L - news + i)  # of the first one's weight
    want = light * v[1] / (1 + light)
    # dS <= (D/16 + 4) 2^-23 s + 2^-22 (|s| + |m|), s = 19.8, as in the restatement; sums of 2^21 equal fp32 numbers
    # by up to 2^15 additions in a row, each off by half a step of a sum that grows: 2^-24 2^15 / 2 of it at most
    ds = (D / 16 + 4 + 4) * 2.0 ** -23 * 19.8
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * (ds + 2.0 ** -21) + 2.0 ** -10) + 2.0 ** -32 * L * v[1].max()
    assert torch.all((o.double().reshape(B, news, G, D) - want).abs() <= tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_weight_of_rows_that_are_not_numbers(fa, D, window):
    """A query row that is no number spoils the weights of the tokens that it sees, and no others."""
    s = Setup(fa, [200, 130], [6, 3], D=D, seed=4)
    s.append_all()
    q = s.queries(2)
    q[2, 1, 5] = float("nan")  # the third of six new tokens, first KV head: slots up to 196
    common = dict(cu=s.d_cu, max_new=6, window=window)
    good = q.clone()
    good[2, 1] = 0
    out = []
    for x in (q.cuda(), good.cuda()):
        lse = fa.kv_attention(x, s.cache, s.d_table, s.d_lens, **common)[1]
        w = torch.zeros((2, s.H, s.M * 64), device="cuda")
        out.append(fa.kv_accumulate(x, lse, w, s.cache, s.d_table, s.d_lens, **common))
    ok(fa)
    spoiled = torch.zeros(out[0].shape, dtype=torch.bool, device="cuda")
    spoiled[0, 0, 197 - window if window else 0:197] = True
    assert torch.all(torch.isnan(out[0][spoiled]))
    assert torch.equal(out[0][~spoiled], out[1][~spoiled])


@pytest.mark.parametrize("n", [100, 1000])  # row by row, page by page
def test_row_offsets_that_do_not_ascend_are_reported(fa, n):
    """Wherever the descent is, or the row that is not there; the other calls see every sequence anyway."""
    s = Setup(fa, [6 * n] * 4, [1] * 4, D=64, seed=3)
    s.append_all()
    ok(fa)
    k = torch.zeros((6 * n, s.H, s.D), dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 5 * n, n, 6 * n, 6 * n], [0, n, 3 * n, 3 * n - 1, 6 * n], [0, 0, n, 6 * n, 5 * n], [n, 0, n, 2 * n, 6 * n],
               [0, n, -1, n, 6 * n], [0, n, 6 * n + 1, n, 6 * n], [0, n, 6 * n, 6 * n, 6 * n + 3]):
        at = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for call in (lambda: fa.kv_append(k, k, s.cache, s.d_table, s.d_lens, cu=at),
                     lambda: fa.kv_read(s.cache, s.d_table, s.d_lens, 6 * n, cu=at)):
            call()
            torch.cuda.synchronize()
            assert fa.device_status() == fa.FP4ATTN_ERR_BAD_INDEX, cu


@pytest.mark.parametrize("n", [3, 1000])
def test_rows_before_the_first_sequence_stay(fa, n):
    """A part of a longer batch: cu begins past 0."""
    s = Setup(fa, [n + 70, n + 30], [n, n], D=64, seed=3)
    s.append_all()
    ok(fa)
    pages = s.cache.pages.clone()
    T = 2 * n + 20
    cu = torch.tensor([11, 11 + n, 11 + 2 * n], dtype=torch.int32, device="cuda")
    want = fa.kv_read(s.cache, s.d_table, s.d_lens, 2 * n)
    out = [torch.full((T, s.H, s.D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.kv_read(s.cache, s.d_table, s.d_lens, T, cu=cu, k=out[0], v=out[1])
    ok(fa)
    for x, y in zip(out, want):
        assert torch.all(x[:11] == 7.0) and torch.all(x[11 + 2 * n:] == 7.0) and torch.equal(x[11:11 + 2 * n], y)
    new = [torch.cat([torch.cat([torch.full((11, s.H, s.D), 9.0)] + [x[b][L - n:].float() for b, L in enumerate(s.lens)])
                      , torch.full((9, s.H, s.D), 9.0)]).bfloat16().cuda() for x in (s.k, s.v)]
    fa.kv_append(new[0], new[1], s.cache, s.d_table, s.d_lens, cu=cu)  # the same rows again
    ok(fa)
    assert torch.equal(s.cache.pages, pages)
    if n == 3:
        q = Setup._bf16(s.rng.standard_normal((T, 4, s.D))).cuda()
        want = fa.kv_attention(q[11:17], s.cache, s.d_table, s.d_lens)
        o, lse = torch.full_like(q, 3.0), torch.full((T, 4), 5.0, device="cuda")
        fa.kv_attention(q, s.cache, s.d_table, s.d_lens, cu=cu, max_new=3, o=o, lse=lse)
        ok(fa)
        assert torch.equal(o[11:17], want[0]) and torch.equal(lse[11:17], want[1])
        assert torch.all(o[:11] == 3.0) and torch.all(o[17:] == 3.0) and torch.all(lse[:11] == 5.0)


def test_one_row_of_one_head_with_any_strides(fa):
    s = Setup(fa, [70], [1], H=1, D=64, seed=6)
    s.append_all()
    ok(fa)
    pages = s.cache.pages.clone()
    odd = [torch.empty_strided((1, 1, 64), (67, 129, 1), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, y in zip(odd, (s.k[0], s.v[0])):
        x.copy_(y[69:70])
    fa.kv_append(odd[0], odd[1], s.cache, s.d_table, s.d_lens)  # the same row again
    a = fa.kv_attention(odd[0], s.cache, s.d_table, s.d_lens)
    b = fa.kv_attention(odd[0].contiguous(), s.cache, s.d_table, s.d_lens)
    ok(fa)
    assert torch.equal(s.cache.pages, pages) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_weights_wider_than_32_bits_count(fa):
    """2^32 + 64 slots (17 GB) are refused like any number above 2^30."""
    s = Setup(fa, [100], [1], H=1, D=64, seed=6)
    s.append_all()
    q = s.queries(1).cuda()
    _, lse = fa.kv_attention(q, s.cache, s.d_table, s.d_lens)
    w = torch.empty((1, 1, 2 ** 32 + 64), device="cuda")
    nt = torch.from_numpy(s.spare[:1].reshape(1, 1).copy()).cuda()
    for call in (lambda: fa.kv_accumulate(q, lse, w, s.cache, s.d_table, s.d_lens),
                 lambda: fa.kv_evict(s.cache, w, s.d_table, s.d_lens, nt, 60)):
        with pytest.raises(fa.Fp4AttnError) as e:
            call()
        assert e.value.status == fa.FP4ATTN_ERR_UNSUPPORTED
    ok(fa)


def test_first_call_of_a_process_in_a_capture_of_a_blocking_stream():
    """While a stream that waits for the legacy one is being captured, nothing may use the legacy stream: the set-up of
    the library's status word does not."""
    import os
    import subprocess
    import sys

    code = """
import ctypes, re
import torch, blackwell_nvfp4_quantize_gb300 as fa
i32 = dict(dtype=torch.int32, device='cuda')
c = fa.empty_kv_cache(4, 2, 64, 'cuda')
k = torch.ones((1, 2, 64), dtype=torch.bfloat16, device='cuda')
table, lens = torch.tensor([[3]], **i32), torch.tensor([1], **i32)
torch.cuda.synchronize()
so = {l.split()[-1] for l in open('/proc/self/maps') if re.search(r'libcudart\\.so', l)}
rt = ctypes.CDLL(so.pop())
st, graph, run = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(st)) == 0
assert rt.cudaStreamBeginCapture(st, 0) == 0
fa.kv_append(k, k, c, table, lens, stream=st.value)
assert rt.cudaStreamEndCapture(st, ctypes.byref(graph)) == 0
assert rt.cudaGraphInstantiate(ctypes.byref(run), graph, ctypes.c_ulonglong(0)) == 0
assert rt.cudaGraphLaunch(run, st) == 0 and rt.cudaStreamSynchronize(st) == 0
a, b = fa.kv_read(c, table, lens, 1)
torch.cuda.synchronize()
assert fa.device_status() == 0 and torch.equal(b, a) and torch.all((a - 1).abs() < 0.1), a
print('done')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr


def plain_attention(fa, s, q, G, cap=0.0, window=0):
    """(O, LSE) in float64 on the GPU, of the values that the cache holds."""
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(s.lens, s.news)):
        one = (s.cache, s.d_table[b:b + 1].contiguous(), s.d_lens[b:b + 1].contiguous())
        k, v = (x.double().repeat_interleave(G, 1) for x in fa.kv_read(*one, L))
        rows = slice(int(s.cu[b]), int(s.cu[b + 1]))
        x = torch.einsum("nhd,lhd->hnl", q[rows].double(), k) * s.D ** -0.5
        if cap:
            x = cap * torch.tanh(x / cap)
        dist = torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")
        x.masked_fill_((dist < 0) | (dist >= window if window else dist < 0), -float("inf"))
        lse[rows] = torch.logsumexp(x, -1).T
        o[rows] = torch.einsum("hnl,lhd->nhd", torch.softmax(x, -1), v)
    return o, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,cap", [(1024, 50.0), (0, 0.0)])
def test_prompts_from_cold_memory(fa, D, window, cap):
    """Problems of two tiles between others of one, so that a tile's warps come to a problem long before its operands,
    which memory delays further; other bytes lie in shared memory at each start."""
    lens, news = [2100, 1500, 1019, 1300], [261, 257, 130, 130]
    s = Setup(fa, lens, news, H=4, D=D, seed=11)
    s.append_all()
    q = s.queries(4).cuda()
    ro, rl = plain_attention(fa, s, q, 4, cap, window)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for turn in range(6):
        flush.fill_(turn)
        o, lse = rows_alone(fa, s, q, softcap=cap, window=window)
        ok(fa)
        # bf16 and fp16 roundings (2^-8 |O| + 2^-11 |V|), and the scores' errors (below 2^-14 here)
        assert torch.all((o.double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -11 + 2.0 ** -13) * 6), turn
        assert torch.all((lse.double() - rl).abs() <= 2.0 ** -14), turn


def test_captured_calls_on_another_stream(fa):
    """A graph whose calls run on a stream that forks off the captured one; their memory belongs to the graph."""
    s = Setup(fa, [700, 190], [1, 1], seed=2, spare=6, columns=WIDE)
    s.append_all()
    q, big = (Setup._bf16(s.rng.standard_normal((n, 4, s.D))).cuda() for n in (2, 100))
    calls = stream_calls(fa, s, q, big)
    want = {n: f(None) for n, f in calls.items() if n != "evict"}
    ok(fa)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = {n: calls[n](side) for n in want}
        torch.cuda.current_stream().wait_stream(side)
        total = sum(x.float().sum() for y in got.values() for x in y)
    for _ in range(3):
        for y in got.values():
            for x in y:
                x.fill_(3)
        graph.replay()
        ok(fa)
        assert all(torch.equal(a, b) for n in want for a, b in zip(got[n], want[n])) and torch.isfinite(total)


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_on_two_streams_beside_other_attention(fa, D):
    """Two prompts at once, each with memory of its own, while a third stream runs the attention of whole tensors."""
    two = [Setup(fa, [1500, 300], [300, 280], H=4, D=D, seed=i) for i in (1, 2)]
    for s in two:
        s.append_all()
    qs = [s.queries(4).cuda() for s in two]
    x = [torch.randn((1, 4, 1024, D), device="cuda").bfloat16() for _ in range(3)]
    want = [rows_alone(fa, s, q) for s, q in zip(two, qs)]
    whole = fa.attention(*x)
    ok(fa)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(15):
        for i, (s, q) in enumerate(zip(two, qs)):
            got[i].append(rows_alone(fa, s, q, stream=streams[i]))
        with torch.cuda.stream(streams[2]):
            got[2].append(fa.attention(*x))
    ok(fa)
    for g, w in zip(got, want + [whole]):
        assert all(torch.equal(a, b) for y in g for a, b in zip(y, w))
