"""Paged cache kernels on the GPU against the 64-bit oracle: map, append, select, attention,
and a run of all four as a serving loop makes it."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_attention_chunk_b200 import build, vkv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vkv.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def new_err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def f64(x):
    return x.detach().to(torch.float32).cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------------------------------------
# map
# ---------------------------------------------------------------------------------------------
def run_map(kv, new, table, ring, pos, page, cap, alias=False, stride=None):
    R, W = table.shape
    err = new_err()
    store = torch.full((R, stride or W), -7, dtype=torch.int32, device=DEV)
    t = store[:, :W]
    t.copy_(torch.from_numpy(table))
    ring_d, kv_d = torch.from_numpy(ring).to(DEV), i32(kv)
    pos_d = torch.tensor(pos, dtype=torch.int64, device=DEV)
    out = None
    if alias:
        out = {"kv_len": kv_d, "ring": pos_d, "slot": torch.empty(cap, dtype=torch.int64, device=DEV)}
    out = vkv.page_map(kv_d, i32(new), t, ring_d, pos_d, page, cap, out=out, err=err)
    torch.cuda.synchronize()
    assert (store[:, W:] == -7).all()
    return {k: v.cpu().numpy() for k, v in out.items()}, t.cpu().numpy(), ring_d.cpu().numpy(), int(err.item())


def check_map(kv, new, table, ring, pos, page, cap, alias=False, stride=None):
    got, t, r, err = run_map(kv, new, table, ring, pos, page, cap, alias, stride)
    try:
        want = oracle.page_map(kv, new, table, ring, pos, page, cap)
        code = 0
    except oracle.paged.Refused as e:
        code = e.code
        want = {"kv_len": np.array(kv), "ring_pos": np.array(pos), "slot": np.full(cap, -1), "row": np.full(cap, -1),
                "pos": np.full(cap, -1), "cu": np.zeros(len(kv) + 1), "table": table, "ring": ring}
    assert err == code
    assert np.array_equal(t, want["table"]) and np.array_equal(r, want["ring"])
    for k, v in got.items():
        assert np.array_equal(v, want["ring_pos" if k == "ring" else k]), k
    return code


def random_step(g, R, page, hi, new_hi, spare=3):
    kv = [int(g.integers(-1, hi + 1)) for _ in range(R)]
    new = [int(g.choice([-1, 0, 1, g.integers(0, new_hi + 1)])) for _ in range(R)]
    pages = lambda n: -(-max(n, 0) // page)  # noqa: E731
    W = max(1, max(pages(max(a, 0) + max(b, 0)) for a, b in zip(kv, new)))
    used = sum(pages(a) for a in kv)
    need = sum(pages(max(a, 0) + b) - pages(a) for a, b in zip(kv, new) if b >= 0)
    N = used + need + spare
    perm = g.permutation(N).astype(np.int32)
    table = np.full((R, W), -1, np.int32)
    at = 0
    for r, a in enumerate(kv):
        table[r, :pages(a)] = perm[at:at + pages(a)]
        at += pages(a)
    n_free = N - used
    taken = int(g.integers(0, 5 * N))
    ring = np.full(N, -1, np.int32)
    for i in range(n_free):
        ring[(taken + i) % N] = perm[used + i]
    return kv, new, table, ring, [taken, taken + n_free], sum(max(b, 0) for b in new)


@pytest.mark.parametrize("R, page, hi, new_hi", [
    (1, 1, 0, 1), (1, 16, 40, 1), (3, 5, 30, 17), (33, 16, 100, 40), (256, 64, 1000, 1), (511, 3, 20, 9), (1500, 7, 50, 4),
    (4096, 16, 90, 6), (7, 128, 5000, 20000)])
@pytest.mark.parametrize("alias", [False, True])
def test_map_random(R, page, hi, new_hi, alias):
    g = np.random.default_rng(R * 1000 + page)
    for rep in range(3):
        kv, new, table, ring, pos, tokens = random_step(g, R, page, hi, new_hi)
        assert check_map(kv, new, table, ring, pos, page, max(1, tokens + int(g.integers(0, 7))), alias,
                         table.shape[1] + rep) == 0


@pytest.mark.parametrize("kv, new, pos, cap, code", [
    ([3], [2], [0, 0], 4, 4), ([3], [6], [0, 6], 4, 4), ([3], [10], [0, 6], 99, 4), ([13], [0], [0, 6], 4, 3),
    ([-2], [0], [0, 6], 4, 3), ([0], [-2], [0, 6], 4, 3), ([0], [1], [5, 4], 4, 3), ([0], [1], [0, 9], 4, 3),
    ([4], [-1], [0, 8], 4, 3), ([0, 2], [2**31 - 1, 2**31 - 1], [0, 6], 4, 4), ([0], [1], [-1, 4], 4, 3)])
@pytest.mark.parametrize("alias", [False, True])
def test_map_refusals(kv, new, pos, cap, code, alias):
    table = np.arange(3 * len(kv), dtype=np.int32).reshape(len(kv), 3)
    assert check_map(kv, new, table, np.arange(8, dtype=np.int32), pos, 4, cap, alias) == code


def test_map_late_ring_positions():
    """Positions past 2^32: a loop that has run for long."""
    big = 7 * (1 << 40) + 5
    assert check_map([3, -1], [9, 4], np.full((2, 4), 1, np.int32), np.arange(11, dtype=np.int32), [big, big + 6], 4,
                     20) == 0


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
def cache_pair(N, P, Hkv, d, kv, g, layout="tokens"):
    """Random cache tensors; layout "heads" has the head axis outside the token axis, "padded" rows apart."""
    def one():
        if layout == "heads":
            x = torch.empty((N, Hkv, P, d), dtype=TYPES[kv], device=DEV).transpose(1, 2)
        elif layout == "padded":
            x = torch.empty((N, P + 1, Hkv + 1, 2 * d), dtype=TYPES[kv], device=DEV)[:, :P, :Hkv, :d]
        else:
            x = torch.empty((N, P, Hkv, d), dtype=TYPES[kv], device=DEV)
        x.copy_(torch.randn((N, P, Hkv, d), device=DEV, generator=g).to(TYPES[kv]))
        return x
    return one(), one()


def bits(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16)


@pytest.mark.parametrize("x, kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("d, Hkv, P", [(64, 1, 16), (128, 8, 64), (128, 3, 5), (64, 12, 1), (128, 2, 200)])
@pytest.mark.parametrize("means", [False, True])
@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
def test_append(x, kv, d, Hkv, P, means, layout):
    gen = torch.Generator(device=DEV).manual_seed(P * 7 + d)
    g = np.random.default_rng(P)
    rows = [(0, 1), (P, 1), (P - 1, 2), (3 % P, 3 * P + 1), (2 * P, 0), (0, 2 * P), (1, 37)]  # (held, new)
    need = [-(-(a + b) // P) for a, b in rows]
    N = sum(need) + 4
    perm = g.permutation(N)
    k, v = cache_pair(N, P, Hkv, d, kv, gen, layout)
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (torch.rand(Hkv, device=DEV, generator=gen) * 0.1 + 0.01 for _ in range(2))
    slot, at, upto = [], 0, {}
    for (a, b), n in zip(rows, need):
        pages = perm[at:at + n]
        at += n
        for t in range(a, a + b):
            slot.append(int(pages[t // P]) * P + t % P)
            upto[int(pages[t // P])] = t % P + 1
    slot += [-1, -1]
    T = len(slot)
    wide = torch.randn((2, T, Hkv + 2, d), device=DEV, generator=gen).to(TYPES[x])
    kn, vn = wide[0, :, :Hkv], wide[1, :, 1:1 + Hkv]
    slot_d = torch.tensor(slot, dtype=torch.int64, device=DEV)
    kbar = torch.full((N, Hkv, d), 9.0, device=DEV) if means else None
    k0, v0 = k.clone(), v.clone()
    err = new_err()
    vkv.page_append(kn, vn, slot_d, k, v, k_scale=ks, v_scale=vs, kbar=kbar, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    live = slot_d >= 0
    for cache, before, new, s in ((k, k0, kn, ks), (v, v0, vn, vs)):
        want = new[live]
        if s is not None:  # fp32 quotient, saturated, rounded once
            want = (want.float() / s[None, :, None]).clamp(-448, 448).to(TYPES[kv])
        flat = before.reshape(N * P, Hkv, d).clone() if layout == "tokens" else before.contiguous().view(N * P, Hkv, d)
        bits(flat)  # same storage
        flat.view(torch.uint8).view(N * P, -1)[slot_d[live]] = want.contiguous().view(torch.uint8).view(int(live.sum()), -1)
        assert torch.equal(bits(cache).view(-1), bits(flat).view(-1))
    if means:
        stored = f64(k)
        scale = np.ones(Hkv) if ks is None else f64(ks)
        got = f64(kbar)
        for page in range(N):
            if page not in upto:
                assert (got[page] == 9.0).all()
                continue
            n = upto[page]
            want = oracle.page_means(stored[page], n) * scale[:, None]
            # n fp32 additions, a division, a product: at most (n + 2) half-ulps of the sum of magnitudes
            tol = (n + 2) * 2.0**-24 * np.abs(stored[page, :n]).mean(0) * scale[:, None]
            assert (np.abs(got[page] - want) <= tol).all()


@pytest.mark.parametrize("means", [False, True])
def test_append_saturates_and_keeps_nan(means):
    k = torch.zeros(2, 4, 1, 64, device=DEV).to(torch.float8_e4m3fn)
    v = k.clone()
    x = torch.zeros(2, 1, 64, device=DEV, dtype=torch.bfloat16)
    x[0, 0, :6] = torch.tensor([1e4, -1e4, float("inf"), -float("inf"), float("nan"), 2.0**-10], device=DEV)
    x[1, 0, :2] = torch.tensor([460.0, 465.0], device=DEV)
    kbar = torch.zeros(2, 1, 64, device=DEV) if means else None
    vkv.page_append(x, x, torch.tensor([4, 5], device=DEV), k, v, kbar=kbar)
    got = k.float()[1]
    assert got[0, 0, :4].tolist() == [448, -448, 448, -448] and got[0, 0, 4].isnan() and got[0, 0, 5] == 0.0
    assert got[1, 0, :2].tolist() == [448, 448]
    if means:
        assert kbar[1, 0, 4].isnan() and kbar[1, 0, 0] == 448.0  # both tokens store 448


@pytest.mark.parametrize("means", [False, True])
def test_append_bad_slots_and_no_tokens(means):
    k = torch.zeros(2, 4, 1, 64, device=DEV, dtype=torch.bfloat16)
    v, err = k.clone(), new_err()
    x = torch.ones(3, 1, 64, device=DEV, dtype=torch.bfloat16)
    kbar = torch.zeros(2, 1, 64, device=DEV) if means else None
    vkv.page_append(x, x, torch.tensor([8, 1 << 40, 2], device=DEV), k, v, kbar=kbar, err=err)
    assert int(err.item()) == vkv.DEVERR_BAD_INDEX
    assert k[0, 2].eq(1).all() and int(k.count_nonzero()) == 64
    err.zero_()
    before = k.clone()
    vkv.page_append(x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device=DEV), k, v, kbar=kbar, err=err)
    assert int(err.item()) == 0 and torch.equal(k, before)


# ---------------------------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("R, H, Hkv, d, P, W, topk, first, last", [
    (1, 1, 1, 64, 16, 1, 1, 0, 0), (3, 8, 2, 128, 16, 40, 7, 1, 2), (5, 40, 8, 128, 64, 300, 64, 2, 4),
    (2, 12, 12, 64, 5, 700, 33, 0, 1), (4, 16, 1, 128, 1, 1500, 97, 3, 3), (2, 10, 2, 64, 128, 20, 128, 0, 0),
    (1, 4, 2, 128, 32, 5000, 4096, 1, 1), (1, 4, 4, 64, 16, 9000, 1, 0, 1)])
@pytest.mark.parametrize("qt", ["bf16", "fp16"])
def test_select(R, H, Hkv, d, P, W, topk, first, last, qt):
    gen = torch.Generator(device=DEV).manual_seed(W + topk)
    g = np.random.default_rng(W)
    N = min(R * W + 3, 20000)
    kbar = torch.randn((N, Hkv, d), device=DEV, generator=gen)
    kbar[N // 2:N // 2 + max(1, N // 8)] = kbar[0]  # many equal scores
    table = i32(g.integers(0, N, (R, W + 2)))[:, :W]
    q = torch.randn((R, H + 1, d), device=DEV, generator=gen).to(TYPES[qt])[:, :H]
    lens = [int(x) for x in g.integers(0, W * P + 1, R)]
    lens[0] = W * P
    if R > 2:
        lens[1], lens[2] = -1, 0
    if R > 3:
        lens[3] = min(W, topk) * P - (P > 1)
    err = new_err()
    sel = vkv.page_select(q, kbar, table, i32(lens), P, topk, first, last, err=err)
    want = oracle.page_select(f64(q), f64(kbar), table.cpu().numpy(), lens, P, topk, first, last)
    assert int(err.item()) == 0
    assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("W", [1500, 2048, 2049, 5000, 8193, 20000])
@pytest.mark.parametrize("scores", ["spread", "few", "equal"])
def test_select_wide_tables(W, scores):
    """Tables of each width that the ranking treats differently, with rows that fill them and rows that
    do not; scores of a handful of values (long runs of ties), or all equal."""
    P, Hkv, d = 2, 2, 64
    gen = torch.Generator(device=DEV).manual_seed(W)
    lens = [W * P, 40 * P, W * P // 3, 0]
    kbar = torch.zeros((300, Hkv, d), device=DEV)
    if scores == "spread":
        kbar.normal_(generator=gen)
    elif scores == "few":
        kbar[:, :, 0] = torch.randint(0, 4, (300, Hkv), device=DEV, generator=gen).float()
    table = torch.randint(0, 300, (len(lens), W), dtype=torch.int32, device=DEV, generator=gen)
    q = torch.rand((len(lens), 4, d), device=DEV, generator=gen).to(torch.bfloat16) + 0.5
    for topk, first, last in ((1, 0, 0), (33, 2, 3), (700, 1, 0)):
        err = new_err()
        sel = vkv.page_select(q, kbar, table, i32(lens), P, topk, first, last, err=err)
        want = oracle.page_select(f64(q), f64(kbar), table.cpu().numpy(), lens, P, topk, first, last)
        assert int(err.item()) == 0 and np.array_equal(sel.cpu().numpy(), want), topk


def test_select_infinities_nan_and_bad_pages():
    N, W, P = 40, 30, 8
    gen = torch.Generator(device=DEV).manual_seed(3)
    kbar = torch.randn((N, 1, 64), device=DEV, generator=gen)
    kbar[3], kbar[4, 0, 0], kbar[5, 0, 0], kbar[6] = float("nan"), float("inf"), -float("inf"), 0.0
    table = i32([list(range(W))])
    table[0, 11], table[0, 12] = N, -1
    q = torch.rand((1, 2, 64), device=DEV, generator=gen).to(torch.bfloat16) + 0.5
    for topk in (1, 5, 26, 27, 28, 29, 30, 31):
        err = new_err()
        sel = vkv.page_select(q, kbar, table, i32([W * P]), P, topk, err=err)
        want = oracle.page_select(f64(q), f64(kbar), table.cpu().numpy(), [W * P], P, topk)
        if topk < W:  # a row whose pages are all kept is not ranked
            assert int(err.item()) == vkv.DEVERR_BAD_INDEX
        assert np.array_equal(sel.cpu().numpy(), want), topk
    err = new_err()
    sel = vkv.page_select(q, kbar, table, i32([W * P + 1]), P, 3, err=err)
    assert int(err.item()) == vkv.DEVERR_BAD_OFFSETS and (sel == -1).all()


def test_select_streams_and_captured_graphs():
    """Calls at the same time on two streams, and two graphs replayed at the same time, do not share scores."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    P, W, topk = 4, 3000, 50
    cases = []
    for i in range(2):
        kbar = torch.randn((500, 4, 64), device=DEV, generator=gen)
        table = torch.randint(0, 500, (6, W), dtype=torch.int32, device=DEV, generator=gen)
        q = torch.randn((6, 8, 64), device=DEV, generator=gen).to(torch.bfloat16)
        cases.append((q, kbar, table, i32([W * P, 900, 0, -1, 5000 + i, 7777]), P, topk, 1, 2))
    want = [vkv.page_select(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(vkv.page_select(*cases[i]))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vkv.page_select(*c))
        graphs.append(g)
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i] + [outs[i]])


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def check_attn(o, lse, ref, q_type, d):
    """o and lse against the oracle's (o, lse, terms).

    A score is a sum of d products in fp32 (each step off by at most 2^-23 of the magnitudes'
    sum A, products included), scaled by two fp32 factors: off by (d + 4) 2^-23 A.  Weights
    exp2 of that: relative error e_w = 2 (d + 4) 2^-23 A + 2^-20 (the exponential), their sum
    over n tokens n 2^-24 more, and what is left of a weight after its two 16-bit parts 2^-16
    (2 x 2^-8 bf16 half-steps).  o is off by at most 2 e_w max|v| plus its own rounding, half a
    step of the output type; the output type's smallest step covers values near zero.
    """
    ro, rl, terms = ref
    A, vmax, n = terms[..., 0], terms[..., 1], terms[..., 2]
    e_w = 2 * (d + 4) * 2.0**-23 * A + 2.0**-20 + n * 2.0**-24
    go, gl = f64(o), f64(lse)
    info = torch.finfo(TYPES[q_type])
    tol = (2 * e_w + 2.0**-15)[..., None] * vmax[..., None] + info.eps / 2 * np.abs(ro) * 1.01 + info.smallest_normal * info.eps
    kept = np.isnan(rl)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(go - ro) <= tol) & ~kept[..., None]
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(go - ro)[bad][:4], tol[bad][:4])
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl) & ~kept, empty)
    live = ~kept & ~empty
    off, at = np.abs(gl[live] - rl[live]), np.abs(rl[live])
    assert (off <= e_w[live] + 2.0**-22 * at + 2.0**-22).all()


def attn_case(R, H, Hkv, d, P, lens, q="bf16", kv="bf16", sink=0, window=0, topk=0, layout="tokens", seed=0, poison=True,
              W=None, q_scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed + P)
    g = np.random.default_rng(seed + P)
    pages = [-(-max(n, 0) // P) for n in lens]
    W = W or max(1, max(pages))
    N = sum(pages) + 3
    perm = g.permutation(N).astype(np.int32)
    table = np.full((R, W), -1, np.int32)
    k, v = cache_pair(N, P, Hkv, d, kv, gen, layout)
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (torch.rand(Hkv, device=DEV, generator=gen) + 0.5 for _ in range(2))
    sel = np.full((R, Hkv, topk), -1, np.int32) if topk else None
    seen = np.zeros((N, P, Hkv), bool)
    at = 0
    for r, n in enumerate(lens):
        table[r, :pages[r]] = perm[at:at + pages[r]]
        at += pages[r]
        for h in range(Hkv):
            toks = oracle.paged.visible_tokens(n, sink, window)
            if topk:
                kept = np.sort(g.permutation(pages[r])[:min(topk, pages[r])])
                sel[r, h, :len(kept)] = kept
                toks = [t for j in kept for t in range(j * P, min(n, j * P + P))]
            for t in toks:
                seen[table[r, t // P], t % P, h] = True
    if poison:  # NaN wherever no query may look
        hole = torch.from_numpy(~seen).to(DEV)
        nan = torch.full((1,), float("nan"), device=DEV).to(k.dtype)
        for c in (k, v):
            c.copy_(torch.where(hole[..., None], nan.float(), c.float()).to(c.dtype))
    qx = (torch.randn((R, H, d), device=DEV, generator=gen) * q_scale).to(TYPES[q])
    return dict(q=qx, k=k, v=v, table=torch.from_numpy(table).to(DEV), lens=lens, ks=ks, vs=vs, sink=sink, window=window,
                sel=None if sel is None else torch.from_numpy(sel).to(DEV), scale=d**-0.5)


def attn_ref(c):
    kk, vv = np.nan_to_num(f64(c["k"])), np.nan_to_num(f64(c["v"]))
    if c["ks"] is not None:
        kk, vv = kk * f64(c["ks"])[:, None], vv * f64(c["vs"])[:, None]
    return oracle.page_attn(f64(c["q"]), kk, vv, c["table"].cpu().numpy(), c["lens"], c["scale"], c["sink"], c["window"],
                            None if c["sel"] is None else c["sel"].cpu().numpy())


def attn_call(c, **kw):
    return vkv.page_attn(c["q"], c["k"], c["v"], c["table"], i32(c["lens"]), scale=c["scale"], sink=c["sink"],
                         window=c["window"], sel=c["sel"], k_scale=c["ks"], v_scale=c["vs"], **kw)


def run_attn(**kw):
    c = attn_case(**kw)
    R, H, d = c["q"].shape
    o = torch.full((R, H, d), 7.0, dtype=c["q"].dtype, device=DEV)
    lse = torch.full((R, H), 5.0, device=DEV)
    err = new_err()
    attn_call(c, err=err, out=(o, lse))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_attn(o, lse, attn_ref(c), kw.get("q", "bf16"), d)
    for r, n in enumerate(c["lens"]):
        if n < 0:
            assert (o[r] == 7.0).all() and (lse[r] == 5.0).all()
    return c, o, lse


TYPE_PAIRS = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")]


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P, lens", [
    (16, [1]), (64, [0]), (16, [15, 16, 17, 31, 32, 33, 0, -1]), (1, [1, 2, 40, -1, 0]), (5, [4, 5, 6, 333]),
    (24, [700, 1]), (128, [127, 128, 129, 1000]), (64, [2000])])
def test_attn_lengths(q, kv, d, P, lens):
    run_attn(R=len(lens), H=6, Hkv=2, d=d, P=P, lens=lens, q=q, kv=kv)


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("H, Hkv", [(1, 1), (2, 1), (5, 1), (8, 1), (9, 1), (12, 3), (16, 1), (17, 1), (40, 1), (24, 2), (40, 8),
                                    (12, 12)])
def test_attn_heads(q, kv, H, Hkv):
    run_attn(R=3, H=H, Hkv=Hkv, d=128, P=32, lens=[70, 301, 5], q=q, kv=kv, seed=H)
    run_attn(R=2, H=H, Hkv=Hkv, d=64, P=32, lens=[40, 133], q=q, kv=kv, seed=H)


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("sink, window", [(0, 1), (0, 100), (1, 1), (17, 45), (300, 300), (1000, 1), (0, 100000), (7, 1000)])
def test_attn_sink_and_window(q, kv, sink, window):
    run_attn(R=4, H=4, Hkv=2, d=128, P=16, lens=[500, 18, 0, 1000], q=q, kv=kv, sink=sink, window=window)


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("P, topk", [(16, 1), (16, 9), (7, 20), (64, 4), (1, 33), (100, 200)])
def test_attn_selected_pages(q, kv, P, topk):
    run_attn(R=5, H=8, Hkv=4, d=128, P=P, lens=[30 * P - P // 2, 3, 0, -1, 9 * P], q=q, kv=kv, topk=topk)
    run_attn(R=2, H=8, Hkv=4, d=64, P=P, lens=[30 * P - P // 2, 3 * P], q=q, kv=kv, topk=topk)


@pytest.mark.parametrize("layout", ["heads", "padded"])
@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
def test_attn_layouts(layout, q, kv):
    run_attn(R=3, H=10, Hkv=2, d=128, P=24, lens=[100, 515, 1], q=q, kv=kv, layout=layout, W=40)


def test_attn_many_rows():
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(-1, 40, 700)]
    run_attn(R=700, H=4, Hkv=2, d=64, P=16, lens=lens)
    run_attn(R=4096, H=2, Hkv=1, d=64, P=8, lens=[(-1, 0, 3, 9)[i % 4] for i in range(4096)])
    run_attn(R=900, H=1, Hkv=1, d=64, P=16, lens=[-1] * 449 + [250] + [-1] * 450)


@pytest.mark.parametrize("H, Hkv, n, kv", [(16, 1, 20011, "bf16"), (8, 1, 60001, "e4m3"), (5, 1, 30000, "bf16")])
def test_attn_long_rows(H, Hkv, n, kv):
    run_attn(R=2, H=H, Hkv=Hkv, d=128, P=64, lens=[n, 700], kv=kv)


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("R, H, Hkv, hi", [(150, 20, 4, 500), (150, 48, 4, 300), (100, 8, 2, 500), (100, 24, 2, 900), (500, 4, 4, 90)])
def test_attn_batches(q, kv, d, R, H, Hkv, hi):
    """Rows times key heads above and below the number of blocks: equal shares that cut rows, and
    whole blocks of more than 32 rows; pairs of key heads where rows are of 128 bytes."""
    g = np.random.default_rng(R + H)
    lens = [int(n) for n in g.integers(-1, hi + 1, R)]
    lens[0], lens[7], lens[R - 1] = hi, 0, -1
    run_attn(R=R, H=H, Hkv=Hkv, d=d, P=16, lens=lens, q=q, kv=kv, seed=R)


@pytest.mark.parametrize("H, Hkv, d, kv, lens", [
    (4, 4, 64, "bf16", [70000, 41, 60000]), (8, 2, 128, "e4m3", [130001, 7, 120000]), (36, 3, 64, "fp16", [64000, 50001]),
    (4, 2, 128, "fp16", [60000, 33, 61111]), (10, 1, 128, "e4m3", [160000, 170001])])
def test_attn_shares_of_long_rows(H, Hkv, d, kv, lens):
    """More tiles per warp than calls of whole blocks have: few rows, cut many times."""
    run_attn(R=len(lens), H=H, Hkv=Hkv, d=d, P=64, lens=lens, q="bf16" if kv != "fp16" else "fp16", kv=kv, poison=False)


def test_attn_all_idle_and_all_empty():
    run_attn(R=3, H=4, Hkv=2, d=64, P=16, lens=[-1, -1, -1])
    run_attn(R=3, H=4, Hkv=2, d=64, P=16, lens=[0, 0, 0])


@pytest.mark.parametrize("q, kv", TYPE_PAIRS)
@pytest.mark.parametrize("q_scale", [1e-6, 30.0, 2000.0])
def test_attn_score_ranges(q, kv, q_scale):
    """From flat softmaxes to ones that a single token wins."""
    run_attn(R=2, H=6, Hkv=2, d=128, P=16, lens=[400, 77], q=q, kv=kv, q_scale=q_scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attn_query_range(kv):
    """bf16 queries outside the range of a 16-bit float with 5 exponent bits."""
    c = attn_case(R=3, H=4, Hkv=2, d=128, P=16, lens=[100, 200, 31], kv=kv)
    for mult in (2.0**90, 2.0**-90):
        q0, s0 = c["q"], c["scale"]
        c["q"], c["scale"] = q0 * mult, s0 / mult
        o, lse = attn_call(c)
        check_attn(o, lse, attn_ref(c), "bf16", 128)
        c["q"], c["scale"] = q0, s0
    c["q"] = c["q"].clone()
    c["q"][1, 1] = 0.0  # one head's query is zero: the mean of the values
    o, lse = attn_call(c)
    check_attn(o, lse, attn_ref(c), "bf16", 128)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attn_nan_and_infinite_queries_stay_with_their_head(kv):
    c = attn_case(R=2, H=6, Hkv=2, d=128, P=16, lens=[100, 50], kv=kv)
    c["q"][0, 1, 5], c["q"][1, 3, 0] = float("nan"), float("inf")
    o, lse = attn_call(c)
    ref = attn_ref({**c, "q": torch.nan_to_num(c["q"], 0.0, 0.0, 0.0)})
    for r, h in ((0, 1), (1, 3)):
        assert o[r, h].isnan().all() and not lse[r, h].isfinite()
        ref[1][r, h] = np.nan  # not compared
    check_attn(o, lse, ref, "bf16", 128)


def test_attn_bad_pages_and_lengths():
    c = attn_case(R=4, H=4, Hkv=2, d=64, P=16, lens=[100, 64, 40, 10])
    N = c["k"].shape[0]
    c["table"][0, 2], c["table"][1, 0] = N, -3
    err = new_err()
    ref = attn_ref(c)  # the oracle skips what such a page holds
    o, lse = attn_call(c, err=err)
    assert int(err.item()) == vkv.DEVERR_BAD_INDEX
    check_attn(o, lse, ref, "bf16", 64)
    W = c["table"].shape[1]
    o.fill_(3.0), lse.fill_(3.0)
    for bad in (W * 16 + 1, -2, -2**31, 2**31 - 1):
        c["lens"] = [100, 64, bad, 10]
        err.zero_()
        attn_call(c, err=err, out=(o, lse))
        assert int(err.item()) in (vkv.DEVERR_BAD_OFFSETS, vkv.DEVERR_BAD_INDEX)
        assert (o[2] == 3.0).all() and (lse[2] == 3.0).all()
        keep = [0, 1, 3]
        check_attn(o[keep], lse[keep], tuple(x[keep] for x in ref), "bf16", 64)
    c["lens"] = [100, 64, 40, 10]
    c["sel"] = i32([[[0, W]], [[1, -1]], [[-1, -1]], [[0, -5]]]).expand(4, 2, 2).contiguous()
    err.zero_()
    o, lse = attn_call(c, err=err)
    assert int(err.item()) == vkv.DEVERR_BAD_INDEX
    s = c["sel"].clone()
    s[s >= W], s[s < 0] = -1, -1
    check_attn(o, lse, attn_ref({**c, "sel": s}), "bf16", 64)


def test_attn_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: pages from both ends."""
    N, P, Hkv, d = 33000, 64, 8, 128  # 2.16e9 elements, 4.3 GB
    k = torch.zeros((N, P, Hkv, d), dtype=torch.bfloat16, device=DEV)
    pages = [N - 1, 0, N - 2, 7]
    gen = torch.Generator(device=DEV).manual_seed(1)
    k[torch.tensor(pages, device=DEV)] = torch.randn((4, P, Hkv, d), device=DEV, generator=gen).to(torch.bfloat16)
    q = torch.randn((1, 16, d), device=DEV, generator=gen).to(torch.bfloat16)
    o, lse = vkv.page_attn(q, k, k, i32([pages]), i32([250]))
    small = k[torch.tensor(pages, device=DEV)].clone()
    ref = oracle.page_attn(f64(q), f64(small), f64(small), np.array([[0, 1, 2, 3]]), [250], d**-0.5)
    check_attn(o, lse, ref, "bf16", d)
    x = torch.randn((2, Hkv, d), device=DEV, generator=gen).to(torch.bfloat16)
    slots = torch.tensor([(N - 1) * P + 60, 3], device=DEV)
    kbar = torch.zeros((N, Hkv, d), device=DEV)
    vkv.page_append(x, x, slots, k, k, kbar=kbar)
    assert torch.equal(k[N - 1, 60], x[0]) and torch.equal(k[0, 3], x[1])
    want = k[N - 1, :61].double().mean(0)
    assert (kbar[N - 1].double() - want).abs().max() <= 63 * 2.0**-24 * k[N - 1].double().abs().max()
    del k, kbar
    torch.cuda.empty_cache()


def test_attn_repeats_bit_for_bit():
    c = attn_case(R=3, H=10, Hkv=2, d=128, P=16, lens=[9000, 17, 4001], poison=False)
    o, lse = attn_call(c)
    for _ in range(5):
        o2, l2 = attn_call(c)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_attn_streams_and_captured_graphs():
    """Calls that overlap: two streams, and two graphs replayed on two streams while an eager call runs."""
    cs = [attn_case(R=2, H=10, Hkv=2, d=128, P=16, lens=[20000 + i, 300 * (i + 1)], poison=False, seed=i) for i in range(3)]
    want = [attn_call(c) for c in cs]
    torch.cuda.synchronize()
    lens = [i32(c["lens"]) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [tuple(torch.empty_like(x) for x in w) for w in want]

    def call(i, **kw):
        c = cs[i]
        return vkv.page_attn(c["q"], c["k"], c["v"], c["table"], lens[i], scale=c["scale"], out=outs[i], **kw)

    for _ in range(5):
        for i, s in enumerate(streams):
            call(i, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        o[0].zero_(), o[1].zero_()
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        call(2)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    # a replay reads the lengths of its time
    lens[0].copy_(i32([77, 0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_attn(*outs[0], attn_ref({**cs[0], "lens": [77, 0]}), "bf16", 128)


def test_attn_workspace_argument():
    c = attn_case(R=1, H=5, Hkv=1, d=64, P=16, lens=[5000], poison=False)
    want = attn_call(c)
    ws = torch.zeros(vkv.vkv_page_attn_workspace_size(5, 1, 64), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = attn_call(c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(vkv.VkvError):
        attn_call(c, workspace=ws[:128])


def test_strides_of_axes_of_one_do_not_count():
    """One row, one head, one page, one token: torch leaves any stride on such an axis."""
    d, P = 64, 16
    c = attn_case(R=1, H=1, Hkv=1, d=d, P=P, lens=[13], poison=False, seed=3)
    want = attn_call(c)

    def odd(x, *strides):
        return x.as_strided(x.shape, strides)

    q = odd(c["q"], 3, 5, 1)
    o, lse = odd(torch.empty_like(c["q"]), 7, 1, 1), torch.empty((1, 1), device=DEV)
    k, v = (odd(c[n], P * d, d, 3, 1) for n in ("k", "v"))
    got = attn_call({**c, "q": q, "k": k, "v": v}, out=(o, lse))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    bar = torch.randn((c["k"].shape[0], 1, d), device=DEV)
    sel = vkv.page_select(q, bar, c["table"], i32([13]), P, 1)
    assert sel.tolist() == [[[0]]]
    x = odd(torch.randn((1, 1, d), device=DEV).to(torch.bfloat16), 1, 3, 1)
    one_k, one_v = (odd(torch.zeros((1, 1, 1, d), dtype=torch.bfloat16, device=DEV), 5, 3, 7, 1) for _ in range(2))
    vkv.page_append(x, x, torch.zeros(1, dtype=torch.int64, device=DEV), one_k, one_v)
    assert torch.equal(bits(one_k).flatten(), bits(x).flatten()) and torch.equal(bits(one_v).flatten(), bits(x).flatten())


def test_outputs_that_overlap_are_refused():
    c = attn_case(R=2, H=4, Hkv=2, d=64, P=16, lens=[20, 5], poison=False)
    lse = torch.empty((2, 4), device=DEV)
    with pytest.raises(ValueError, match="o must not be q"):
        attn_call(c, out=(c["q"], lse))
    with pytest.raises(ValueError, match="overlaps itself"):
        attn_call(c, out=(torch.empty_like(c["q"][:1]).expand(2, 4, 64), lse))
    x, slot = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="overlaps itself"):
        vkv.page_append(x, x, slot, c["k"][:1].expand(c["k"].shape), c["v"])
    n = i32([0, 0])
    out = {"kv_len": n, "ring": torch.empty(2, dtype=torch.int64, device=DEV),
           "slot": torch.empty(4, dtype=torch.int64, device=DEV)}
    with pytest.raises(ValueError, match="must not be new_len"):
        vkv.page_map(i32([0, 0]), n, i32([[0], [0]]), i32([0]), torch.zeros(2, dtype=torch.int64, device=DEV), 16, 4, out=out)


# ---------------------------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kv, captured", [("bf16", False), ("e4m3", False), ("bf16", True)])
def test_serving_loop(kv, captured):
    """Requests start, decode, end and start again; every step's cache, means, selection and
    attention against the oracle's own bookkeeping of whole sequences."""
    R, H, Hkv, d, P, W, N, cap, topk = 4, 8, 2, 64, 8, 24, 40, 60, 5
    gen = torch.Generator(device=DEV).manual_seed(11)
    steps = [[9, 30, 0, 0], [1, 1, 0, 17], [1, 1, 5, 1], [1, -1, 1, 1], [1, 0, 1, 1], [20, 21, 1, -1], [1, 1, 1, 2], [-1, 1, -1, 8]]
    table = torch.full((R, W), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(N, device=DEV, generator=gen).to(torch.int32)
    ring_pos = torch.tensor([0, N], dtype=torch.int64, device=DEV)
    kv_len, new_len = torch.full((R,), -1, dtype=torch.int32, device=DEV), i32([0] * R)
    k, v = (torch.zeros((N, P, Hkv, d), device=DEV).to(TYPES[kv]) for _ in range(2))
    for c in (k, v):
        bits(c).fill_(127)  # NaN in e4m3; whatever in bf16: no one may read it
    kbar = torch.full((N, Hkv, d), float("nan"), device=DEV)
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (torch.rand(Hkv, device=DEV, generator=gen) * 0.02 + 0.01 for _ in range(2))
    kn, vn = (torch.zeros((cap, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((R, H, d), dtype=torch.bfloat16, device=DEV)
    out = {"kv_len": kv_len, "ring": ring_pos, "slot": torch.empty(cap, dtype=torch.int64, device=DEV),
           "row": torch.empty(cap, dtype=torch.int32, device=DEV), "pos": torch.empty(cap, dtype=torch.int32, device=DEV)}
    sel = torch.empty((R, Hkv, topk), dtype=torch.int32, device=DEV)
    full, part = ((torch.zeros((R, H, d), dtype=torch.bfloat16, device=DEV), torch.zeros((R, H), device=DEV)) for _ in range(2))
    err = new_err()

    def step():
        vkv.page_map(kv_len, new_len, table, ring, ring_pos, P, cap, out=out, err=err)
        vkv.page_append(kn, vn, out["slot"], k, v, k_scale=ks, v_scale=vs, kbar=kbar, err=err)
        vkv.page_select(q, kbar, table, kv_len, P, topk, 1, 1, err=err, out=sel)
        vkv.page_attn(q, k, v, table, kv_len, k_scale=ks, v_scale=vs, err=err, out=full)
        vkv.page_attn(q, k, v, table, kv_len, sel=sel, k_scale=ks, v_scale=vs, err=err, out=part)

    graph = None
    if captured:  # with no tokens and no requests: nothing changes
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    held = [None] * R  # each request's (keys, values) so far, as stored
    for i, new in enumerate(steps):
        new_len.copy_(i32(new))
        for x in (kn, vn, q):
            x.copy_(torch.randn(x.shape, device=DEV, generator=gen).to(x.dtype))
        for x, _ in (full, part):
            x.fill_(7.0)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        stored = []
        for x, s in ((kn, ks), (vn, vs)):
            y = x if s is None else (x.float() / s[None, :, None]).clamp(-448, 448).to(TYPES[kv])
            stored.append(f64(y) if s is None else f64(y) * f64(s)[:, None])
        at = 0
        for r, n in enumerate(new):
            if n < 0:
                held[r] = None
            elif n > 0:
                old = held[r] or [np.zeros((0, Hkv, d))] * 2
                held[r] = [np.concatenate([a, b[at:at + n]]) for a, b in zip(old, stored)]
                at += n
        lens = [-1 if h is None else len(h[0]) for h in held]
        assert kv_len.tolist() == lens
        # the oracle's cache: row r's page j is page r * W + j
        ck, cv, cm = np.zeros((R * W, P, Hkv, d)), np.zeros((R * W, P, Hkv, d)), np.zeros((R * W, Hkv, d))
        ct = np.arange(R * W).reshape(R, W)
        got_bar = f64(kbar)
        for r, h in enumerate(held):
            for t in range(lens[r]):
                ck[r * W + t // P, t % P], cv[r * W + t // P, t % P] = h[0][t], h[1][t]
            for j in range(-(-lens[r] // P)):
                n = min(P, lens[r] - j * P)
                cm[r * W + j] = oracle.page_means(ck[r * W + j], n)
                mine = got_bar[int(table[r, j])]
                assert (np.abs(mine - cm[r * W + j]) <= (n + 3) * 2.0**-24 * np.abs(ck[r * W + j]).max(0)).all()
                cm[r * W + j] = mine  # rank by the same means
        want = oracle.page_select(f64(q), cm, ct, lens, P, topk, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want)
        check_attn(*full, oracle.page_attn(f64(q), ck, cv, ct, lens, d**-0.5), "bf16", d)
        check_attn(*part, oracle.page_attn(f64(q), ck, cv, ct, lens, d**-0.5, sel=want), "bf16", d)
        for r, n in enumerate(lens):
            if n < 0:
                assert (full[0][r] == 7.0).all() and (part[0][r] == 7.0).all()
    live = [int(p) for r in range(R) for p in table[r, :-(-max(lens[r], 0) // P)]]
    t0, t1 = (int(x) for x in ring_pos)
    free = [int(ring[t % N]) for t in range(t0, t1)]
    assert sorted(live + free) == list(range(N))  # no page lost or held twice
