"""Paged cache kernels on the GPU: calls at the edges of what the documentation allows."""
import threading

import numpy as np
import pytest
import torch

import oracle
from kv_cache_attention_chunk_b200 import build, vkv
from test_gpu_paged import DEV, TYPES, attn_call, attn_case, attn_ref, bits, check_attn, f64, i32, new_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vkv.lib()


def test_attn_refuses_an_empty_selection():
    """A selection of no entries has no address: it must not be taken for no selection."""
    c = attn_case(R=2, H=4, Hkv=2, d=64, P=16, lens=[40, 5], poison=False)
    for sel in (torch.empty((2, 2, 0), dtype=torch.int32, device=DEV), i32(np.zeros((2, 2, 3)).tolist())[:, :, :0]):
        for window in (0, 7):
            with pytest.raises(ValueError, match="sel"):
                attn_call({**c, "sel": sel, "window": window})


@pytest.mark.parametrize("x", ["bf16", "fp16"])
@pytest.mark.parametrize("means", [False, True])
def test_append_e4m3_keeps_the_sign_of_zero(x, means):
    """x / scale is -0 for x = -0 (and for +0 over a negative scale), and e4m3 has both zeros."""
    scale = torch.tensor([0.5, 0.3, 3.0, 2.0**-70, -0.7, 1.0], device=DEV)
    new = torch.zeros((3, 6, 64), dtype=TYPES[x], device=DEV)
    new[:, :, ::3] = -0.0
    new[1, :, 5] = -6.0e-8  # a quotient that rounds to -0 (or not, over a small scale)
    k, v = (torch.ones((2, 4, 6, 64), device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    kbar = torch.zeros((2, 6, 64), device=DEV) if means else None
    vkv.page_append(new, new, torch.tensor([4, 5, 6], device=DEV), k, v, k_scale=scale, v_scale=scale, kbar=kbar)
    want = (new.float() / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert int((bits(want) == 0x80).sum()) > 100
    for got in (k, v):
        assert torch.equal(bits(got[1, :3]), bits(want))


@pytest.mark.parametrize("d", [64, 128])
def test_attn_bf16_values_near_the_largest(d):
    """A finite output of bf16 values near the type's largest: weights stay at 1 or below, also
    where a score exceeds the running maximum by less than what moves it."""
    R, Hkv, P, n = 8, 8, 16, 2048
    N = R * n // P
    k, v = (torch.zeros((N, P, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.arange(N, dtype=torch.int32, device=DEV).view(R, n // P)
    for r in range(R):
        for h in range(Hkv):  # one token with a score of 2.08 among zeros, at another place in each row and head
            t = 40 + 16 * (r * Hkv + h)
            k[table[r, t // P], t % P, h, 0] = 2.078125
            v[table[r, t // P], t % P, h] = 3.0e38 * (-1) ** h
    q = torch.zeros((R, Hkv, d), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    o, lse = vkv.page_attn(q, k, v, table, i32([n] * R), scale=1.0)
    assert o.isfinite().all()
    ref = oracle.page_attn(f64(q), f64(k), f64(v), table.cpu().numpy(), [n] * R, 1.0)
    check_attn(o, lse, ref, "bf16", d)


def test_map_from_several_threads_with_different_row_counts():
    """Calls with more rows than 48 KB of shared memory hold, from several threads at once."""
    failed = []

    def loop(R):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            kv, new = torch.zeros(R, dtype=torch.int32, device=DEV), torch.ones(R, dtype=torch.int32, device=DEV)
            table, ring = torch.full((R, 1), -1, dtype=torch.int32, device=DEV), torch.arange(R, dtype=torch.int32, device=DEV)
            pos, slot = torch.tensor([0, R], device=DEV), torch.zeros(R, dtype=torch.int64, device=DEV)
            kv_out, pos_out = torch.empty_like(kv), torch.empty_like(pos)
            a = vkv.vkv_page_map_args(R, 1, 16, R, R, 0)
            a.kv_len, a.new_len, a.table, a.table_stride = kv.data_ptr(), new.data_ptr(), table.data_ptr(), 1
            a.ring, a.ring_pos, a.kv_len_out, a.ring_pos_out = (x.data_ptr() for x in (ring, pos, kv_out, pos_out))
            a.slot = slot.data_ptr()
            stream.synchronize()
            got = [vkv.vkv_page_map(a, stream.cuda_stream) for _ in range(3000)]
            stream.synchronize()
            if any(got) or not torch.equal(slot, 16 * torch.arange(R, device=DEV)):
                failed.append((R, sum(map(bool, got))))

    threads = [threading.Thread(target=loop, args=(R,)) for R in (4096, 3200, 3900, 3300, 4000, 3100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_select_checks_the_pages_of_short_rows():
    """A row whose pages are all kept is not ranked, but a page number outside the cache is still reported."""
    N, P, W = 9, 4, 6
    kbar, q = torch.ones((N, 3, 64), device=DEV), torch.ones((3, 3, 64), dtype=torch.bfloat16, device=DEV)
    for bad in (-1, N, -(2**31)):
        for row, col in ((0, 0), (0, 2), (2, 3)):
            table = torch.zeros((3, W), dtype=torch.int32, device=DEV)
            table[row, col] = bad
            for topk in (4, 6, 9):  # fewer than the table's columns: some other row could be ranked
                err = new_err()
                sel = vkv.page_select(q, kbar, table, i32([9, 0, 13]), P, topk, err=err)
                assert int(err.item()) == vkv.DEVERR_BAD_INDEX
                assert sel[0, 1].tolist() == [0, 1, 2] + [-1] * (topk - 3)
                assert sel[2, 2].tolist() == [0, 1, 2, 3] + [-1] * (topk - 4)
    table = torch.zeros((3, W), dtype=torch.int32, device=DEV)
    table[0, 3:], table[1], table[2, 4:] = -1, -1, N  # columns behind the rows' pages are not looked at
    for topk in (4, 6, 9):
        err = new_err()
        vkv.page_select(q, kbar, table, i32([9, 0, 13]), P, topk, err=err)
        assert int(err.item()) == 0


def _calls(stream):
    """Each call that makes its outputs itself, with its inputs ready: name -> (call, its outputs' expected values)."""
    c = attn_case(R=2, H=8, Hkv=2, d=128, P=16, lens=[900, 33], poison=False)
    kbar = torch.randn((c["k"].shape[0], 2, 128), device=DEV)
    lens, one = i32(c["lens"]), i32([1, 1])
    n = c["k"].shape[0]
    table, ring, pos = torch.full((2, 4), 7, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV), \
        torch.tensor([0, n], device=DEV)
    kv = i32([3, 5])
    return {"attn": lambda **k: list(vkv.page_attn(c["q"], c["k"], c["v"], c["table"], lens, **k)),
            "select": lambda **k: [vkv.page_select(c["q"], kbar, c["table"], lens, 16, 5, 1, 1, **k)],
            "map": lambda **k: list(vkv.page_map(kv, one, table, ring, pos, 16, 2000, **k).values())}


@pytest.mark.parametrize("name", ["attn", "select", "map"])
def test_outputs_made_for_another_stream(name):
    """Outputs that a call makes for `stream` are memory that no pending work of the current stream still
    writes, and freeing them does not hand them out while the current stream still reads them."""
    s = torch.cuda.Stream()
    call = _calls(s)[name]
    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    got = call(stream=s)  # workspaces and the like exist from here on
    torch.cuda.synchronize()
    del got
    for _ in range(2):
        torch.cuda._sleep(20_000_000)
        junk = [torch.full_like(x, 99) for x in want]  # pending on the current stream, then free for its next allocations
        del junk
        got = call(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copies = [x.clone() for x in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full_like(x, 99) for x in want]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    del junk


def test_append_refuses_keys_and_values_in_one_place():
    x, y = (torch.randn((3, 4, 64), device=DEV).to(torch.bfloat16) for _ in range(2))
    slot = torch.tensor([0, 1, 9], device=DEV)
    buf = torch.zeros((6, 2, 8, 8, 64), dtype=torch.bfloat16, device=DEV)
    one, other = buf[:, 0, :, :4], buf[:, 1, :, :4]
    for k, v, why in ((one, one, "one tensor"), (buf[:, 0, :, :4], buf[:, 0, :, 2:6], "heads in common"),
                      (buf[:5, 0, :, :4], buf[1:, 0, :, :4], "pages in common")):
        with pytest.raises(ValueError, match="overlap"):
            vkv.page_append(x, y, slot, k, v)
        assert int(buf.count_nonzero()) == 0, why
    flat = torch.zeros((7, 8, 4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        vkv.page_append(x, y, slot, flat[:6], flat[1:])
    with pytest.raises(ValueError, match="overlap"):  # the same rows, stored by different scales
        e = torch.zeros((6, 8, 4, 64), device=DEV).to(torch.float8_e4m3fn)
        vkv.page_append(x, x, slot, e, e, k_scale=torch.ones(4, device=DEV), v_scale=torch.full((4,), 2.0, device=DEV))
    store = torch.zeros(6 * 8 * 4 * 64 * 2, dtype=torch.float32, device=DEV)
    k = store[:6 * 8 * 4 * 32].view(torch.bfloat16).view(6, 8, 4, 64)
    with pytest.raises(ValueError, match="kbar overlaps"):
        vkv.page_append(x, y, slot, k, flat[:6], kbar=store[64:64 + 6 * 4 * 64].view(6, 4, 64))
    # side by side in one buffer, by page, by token and by head
    slot = torch.tensor([0, 1, 3], device=DEV)
    for k, v in ((one, other), (buf[:3, 0, :, :4], buf[3:, 0, :, :4]), (buf[:, 0, ::2, :4], buf[:, 0, 1::2, :4]),
                 (buf[:, 0, :, :4], buf[:, 0, :, 4:])):
        buf.zero_()
        vkv.page_append(x, y, slot, k, v)
        assert torch.equal(k[0, slot], x) and torch.equal(v[0, slot], y)
        assert int(buf.count_nonzero()) == int(x.count_nonzero() + y.count_nonzero())
    slot = torch.tensor([0, 1, 9], device=DEV)
    vkv.page_append(x, x, slot, flat[:6], flat[:6])  # one tensor, equal rows
    assert torch.equal(flat[1, 1], x[2])


def test_attn_refuses_outputs_that_lie_in_inputs():
    R, H, d = 3, 4, 64
    c = attn_case(R=R, H=H, Hkv=2, d=d, P=16, lens=[20, 5, 40], poison=False)
    lse = torch.empty((R, H), device=DEV)
    buf = torch.zeros((R + 1, 2 * H, d), dtype=torch.bfloat16, device=DEV)
    for q, o in ((buf[:R, :H], buf[1:, :H]), (buf[:R, :H], buf[:R, 2:2 + H]), (buf[:R, :H], buf[:R, :H])):
        with pytest.raises(ValueError, match="o must not be q|o overlaps q"):
            attn_call({**c, "q": q}, out=(o, lse))
    with pytest.raises(ValueError, match="o overlaps"):
        attn_call(c, out=(c["k"].view(-1)[64:64 + R * H * d].view(R, H, d), lse))
    with pytest.raises(ValueError, match="o overlaps"):
        attn_call(c, out=(c["v"].view(-1)[:R * H * d].view(R, H, d), lse))
    o = torch.empty((R, H, d), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="lse overlaps"):
        attn_call(c, out=(o, o.view(-1)[:2 * R * H].view(torch.float32).view(R, H)))
    with pytest.raises(ValueError, match="lse overlaps"):
        attn_call(c, out=(o, c["q"].view(-1)[:2 * R * H].view(torch.float32).view(R, H)))
    want = attn_call(c)
    buf[:R, :H] = c["q"]  # side by side in one buffer
    attn_call({**c, "q": buf[:R, :H]}, out=(buf[:R, H:], lse))
    assert torch.equal(buf[:R, H:], want[0]) and torch.equal(lse, want[1])


def test_map_refuses_arrays_that_overlap():
    R, W, n, cap = 4, 3, 12, 8

    def call(**kw):
        big = torch.zeros(200, dtype=torch.int32, device=DEV)
        a = {"kv_len": big[:R], "new_len": big[10:10 + R], "table": big[20:20 + R * W].view(R, W), "ring": big[40:40 + n],
             "ring_pos": big[60:64].view(torch.int64), "out_len": big[70:70 + R], "out_ring": big[80:84].view(torch.int64),
             "slot": big[90:90 + 2 * cap].view(torch.int64), "row": big[110:110 + cap], "pos": big[120:120 + cap],
             "cu": big[130:131 + R]}
        a.update({k: f(big) for k, f in kw.items()})
        big[60:64].view(torch.int64)[1] = n
        out = {"kv_len": a["out_len"], "ring": a["out_ring"], "slot": a["slot"], "row": a["row"], "pos": a["pos"], "cu": a["cu"]}
        return vkv.page_map(a["kv_len"], a["new_len"], a["table"], a["ring"], a["ring_pos"], 16, cap, out=out)

    call()
    call(out_len=lambda b: b[:R], out_ring=lambda b: b[60:64].view(torch.int64))  # in place
    wide = lambda b: b[140:140 + R * 8].view(R, 8)[:, :W]  # noqa: E731
    call(table=wide)
    call(table=wide, cu=lambda b: b[143:144 + R])  # between two of the table's rows
    for kw in (dict(out_len=lambda b: b[1:1 + R]), dict(out_len=lambda b: b[9:9 + R]), dict(slot=lambda b: b[78:78 + 2 * cap].view(torch.int64)),
               dict(pos=lambda b: b[112:112 + cap]), dict(cu=lambda b: b[2:3 + R]), dict(ring=lambda b: b[24:24 + n]),
               dict(row=lambda b: b[44:44 + cap]), dict(out_ring=lambda b: b[62:66].view(torch.int64)),
               dict(table=wide, cu=lambda b: b[150:151 + R]), dict(table=wide, cu=lambda b: b[144:145 + R])):
        with pytest.raises(ValueError, match="overlap"):
            call(**kw)


def append_dispatch(T, Hkv, P):
    """(four warps per run, tokens per block) of an append with means, as its launch chooses them."""
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    split = T * Hkv <= 8 * n_sm or P >= 64
    return split, min(32, max(1, T * Hkv // ((16 if split else 64) * n_sm)))


@pytest.mark.parametrize("x, kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("d, Hkv, P, tokens, split, slab", [
    (64, 5, 5, 2100, False, 1), (128, 3, 16, 18000, False, 5), (128, 12, 32, 9000, False, 11), (64, 12, 16, 27000, False, 32),
    (128, 5, 33, 64000, False, 32), (64, 3, 1, 20000, False, 6), (128, 3, 64, 13000, True, 16), (64, 12, 200, 7000, True, 32)])
def test_append_means_of_long_prompts(x, kv, d, Hkv, P, tokens, split, slab):
    """Prompts that start inside a page, runs that cross the blocks' slabs, several runs per slab, idle warps."""
    gen = torch.Generator(device=DEV).manual_seed(P + d)
    g = np.random.default_rng(P)
    held, new = [], []
    while sum(new) < tokens:
        held.append(int(g.integers(0, 2 * P + 1)))
        new.append(int(g.choice([1, g.integers(0, 2 * P + 2), g.integers(0, tokens // 5)])))
    T = sum(new) + 2 * len(new)  # two skipped tokens behind each row's
    got_split, got_slab = append_dispatch(T, Hkv, P)
    assert got_split == split and abs(got_slab - slab) <= max(1, slab // 4)
    pages = [-(-(a + b) // P) for a, b in zip(held, new)]
    N = sum(pages) + 2
    perm = torch.from_numpy(g.permutation(N)).to(DEV)
    slot, upto, at = [], torch.zeros(N, dtype=torch.int64, device=DEV), 0
    for a, b, n in zip(held, new, pages):
        t = torch.arange(a, a + b, device=DEV)
        own = perm[at:at + n]
        at += n
        slot += [own[t // P] * P + t % P, torch.full((2,), -1, device=DEV)]
        upto.scatter_reduce_(0, own[t // P], t % P + 1, "amax")
    slot = torch.cat(slot)
    k, v = (torch.randn((N, P, Hkv, d), device=DEV, generator=gen).to(TYPES[kv]) for _ in range(2))
    kn, vn = (torch.randn((T, Hkv, d), device=DEV, generator=gen).to(TYPES[x]) for _ in range(2))
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (torch.rand(Hkv, device=DEV, generator=gen) * 0.1 + 0.01 for _ in range(2))
    kbar = torch.full((N, Hkv, d), 9.0, device=DEV)
    live = slot >= 0
    want = []
    for cache, rows, s in ((k, kn, ks), (v, vn, vs)):
        w = rows[live] if s is None else (rows[live].float() / s[None, :, None]).clamp(-448, 448).to(TYPES[kv])
        w0 = cache.clone()
        bits(w0).view(N * P, -1)[slot[live]] = bits(w).view(int(live.sum()), -1)
        want.append(w0)
    err = new_err()
    vkv.page_append(kn, vn, slot, k, v, k_scale=ks, v_scale=vs, kbar=kbar, err=err)
    assert int(err.item()) == 0
    assert torch.equal(bits(k), bits(want[0])) and torch.equal(bits(v), bits(want[1]))
    inside = (torch.arange(P, device=DEV)[None] < upto[:, None])[..., None, None]
    stored = torch.where(inside, k.double(), 0.0)
    n = upto.clamp(min=1).double()[:, None, None]
    scale = (torch.ones(Hkv, device=DEV) if ks is None else ks).double()[None, :, None]
    # n fp32 additions, a division, a product: at most (n + 2) half-ulps of the sum of magnitudes
    tol = (n + 2) * 2.0**-24 * stored.abs().sum(1) / n * scale
    off = (kbar.double() - stored.sum(1) / n * scale).abs()
    written = upto > 0
    assert (off[written] <= tol[written]).all() and (kbar[~written] == 9.0).all()


@pytest.mark.parametrize("R, H, Hkv, W, steps", [(3, 4, 2, 2900, 1), (6, 10, 5, 6000, 10), (5, 9, 9, 9001, 16), (64, 24, 12, 700, 16)])
def test_select_several_steps_per_warp(R, H, Hkv, W, steps):
    """d = 128, by the number of steps that a warp of the score kernel takes; rows that end inside a step."""
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    assert min(16, -(-R * Hkv * -(-W // 8) // (16 * n_sm))) == steps
    P, d = 2, 128
    gen = torch.Generator(device=DEV).manual_seed(W)
    lens = [W * P - i % 16 * 37 for i in range(R)]
    lens[1] = 40 * P - 1
    kbar = torch.randn((300, Hkv, d), device=DEV, generator=gen)
    table = torch.randint(0, 300, (R, W), dtype=torch.int32, device=DEV, generator=gen)
    q = torch.randn((R, H, d), device=DEV, generator=gen).to(torch.bfloat16)
    for topk, first, last in ((33, 2, 3),):
        err = new_err()
        sel = vkv.page_select(q, kbar, table, i32(lens), P, topk, first, last, err=err)
        few = [0, 1, 2, R - 1] if R > 16 else list(range(R))
        want = oracle.page_select(f64(q[few]), f64(kbar), table[few].cpu().numpy(), [lens[r] for r in few], P, topk, first, last)
        assert int(err.item()) == 0 and np.array_equal(sel[few].cpu().numpy(), want)


@pytest.mark.parametrize("q, kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("H, Hkv, d, lens", [(6, 2, 128, [400, 77]), (8, 8, 64, [5000, 2003, 33]), (12, 1, 128, [9001]), (3, 1, 64, [30011, 1])])
def test_attn_scores_far_apart(q, kv, H, Hkv, d, lens):
    """Softmaxes that one or few tokens win, maxima that move often and lie far apart where parts are joined.

    q, k and the scales are small whole numbers (times powers of two), so a score s is exact.  Its
    log2 form x, |x| <= X, carries at most 3 x 2^-24 X from c's rounding, the product and the maximum's
    subtraction, so a weight is off by e = 3 x 2^-24 X + 2^-21 (the exponential).  A move of the maximum
    multiplies what came before by one more such factor, but shrinks it 2^4 times at least, and a part's
    weight in the joins is one more: 4 e in all.  The sum over n tokens adds n 2^-24, a weight's two
    16-bit parts leave 2^-16.
    """
    c = attn_case(R=len(lens), H=H, Hkv=Hkv, d=d, P=16, lens=lens, q=q, kv=kv)
    gen = torch.Generator(device=DEV).manual_seed(H)
    whole = lambda t: torch.randint(-3, 4, t.shape, device=DEV, generator=gen).to(t.dtype)  # noqa: E731
    holes = c["k"].float().isnan()
    c["q"] = whole(c["q"])
    c["k"] = torch.where(holes, float("nan"), whole(c["k"]).float()).to(c["k"].dtype)
    c["scale"] = 0.5
    if c["ks"] is not None:
        c["ks"] = torch.tensor([2.0 ** (i % 3 - 1) for i in range(Hkv)], device=DEV)
    o, lse = attn_call(c)
    ro, rl, terms = attn_ref(c)
    X, vmax, n = 1.45 * terms[..., 0] + 16, terms[..., 1], terms[..., 2]
    e_w = 4 * (3 * 2.0**-24 * X + 2.0**-21) + n * 2.0**-24
    info = torch.finfo(TYPES[q])
    tol = (2 * e_w + 2.0**-15)[..., None] * vmax[..., None] + info.eps / 2 * np.abs(ro) * 1.01
    assert (tol < 0.02 * vmax[..., None]).all()  # a wrong row of values does not pass
    assert (np.abs(f64(o) - ro) <= tol).all()
    assert (np.abs(f64(lse) - rl) <= e_w + 2.0**-22 * np.abs(rl) + 2.0**-22).all()
