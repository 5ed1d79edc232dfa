"""Calls on another stream than the current one: the memory that the wrappers make for them."""
import pytest
import torch

from kv_cache_attention_chunk_b200 import build, vkv, workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vkv.lib()


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x] if x.is_cuda else []
    if isinstance(x, dict):
        x = x.values()
    return [t for y in x for t in tensors(y)] if isinstance(x, (list, tuple, type({}.values()))) else []


def apart(x):
    """`x` with a gap behind each element: the wrapper has to make a contiguous copy."""
    return torch.stack([x, torch.zeros_like(x)], -1)[..., 0]


def calls(name):
    if name == "segments":
        c = W.cfg_tiny()
        q, k, v = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV)
        return lambda **kw: vkv.chunk_attn_segments(q, k, v, c.branches, scale=c.scale, **kw)
    if name == "ragged":
        c = W.make_ragged("streams", seed=3, H=4, frame_tokens=64, hist_frames=12, q_frames=2,
                          policies=[("anchor", 3), ("wave", 2), ("veil", 0), ("wave", 3)])
        q, k, v, cu = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), torch.from_numpy(c.cu_seqlens).to(DEV)
        return lambda **kw: vkv.chunk_attn_ragged(q, k, v, cu, c.cu_seqlens, scale=c.scale, **kw)
    if name == "merge":
        a = [x.to(DEV) for x in W.make_merge_inputs(3, 1, 300, 4, 128)]
        return lambda **kw: vkv.lse_merge(*a, **kw)
    if name == "latent":
        c = W.make_latent("streams", seed=1, B=1, H=2, Lq=200, Lkv=300)
        q, kv = c.q.to(DEV), c.kv.to(DEV)
        return lambda **kw: vkv.latent_attn(q, kv, c.d_c, scale=c.scale, **kw)
    if name == "compact":
        g = torch.Generator(device=DEV).manual_seed(5)
        k, v = (torch.randn((1, 12 * 64, 3, 128), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        rules = [(vkv.HEAD_ANCHOR, 3), (vkv.HEAD_WAVE, 2), (vkv.HEAD_FULL, 1)]
        return lambda **kw: vkv.compact_cache(k, v, rules, 64, 10, 2, 2, **kw)[:3]
    c = W.make_block_sparse("streams", seed=5, H=2, d=128, frame_tokens=256, block=64, hist_frames=3, win_frames=4,
                            q_frames=2, n_persist=5)
    q, k, v = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV)
    persist = apart(torch.from_numpy(c.persist_idx).to(DEV))
    if name == "pool":
        return lambda **kw: vkv.block_pool(k, c.window_blk0, c.n_win_blk, **kw)
    kbar = vkv.block_pool(k, c.window_blk0, c.n_win_blk)
    if name == "select":
        means = apart(kbar)
        return lambda **kw: vkv.block_select(q, k, c.window_blk0, c.n_win_blk, 3, scores=True, order=True, kbar=means, **kw)
    sel, _, order = vkv.block_select(q, k, c.window_blk0, c.n_win_blk, 3, order=True)
    if name == "order":
        picked = apart(sel)
        return lambda **kw: vkv.block_order(picked, **kw)
    if name == "persist":
        return lambda **kw: vkv.persist_update(q, k, persist, c.window_blk0, 4, scores=True, **kw)
    sel, order = apart(sel), apart(order)
    return lambda **kw: vkv.chunk_attn_block_sparse(q, k, v, persist, sel, c.window_blk0, c.n_win_blk, scale=c.scale,
                                                    qblk_order=order, **kw)


@pytest.mark.parametrize("name", ["segments", "ragged", "merge", "latent", "compact", "pool", "select", "order", "persist", "sparse"])
def test_memory_made_for_another_stream(name):
    """What a call makes for `stream` (outputs, copies of strided inputs, workspaces) is memory that no pending work
    of the current stream still writes, and freeing it does not hand it out while it is still in use."""
    s = torch.cuda.Stream()
    call = calls(name)
    want = [x.clone() for x in tensors(call())]
    assert want
    torch.cuda.synchronize()
    sizes = [x.numel() * x.element_size() for x in want] + [512 << i for i in range(12)]

    def junk():
        return [torch.full((n,), 1, dtype=torch.uint8, device=DEV) for n in sizes]

    for _ in range(2):
        torch.cuda._sleep(20_000_000)
        pending = junk()  # still to be written on the current stream, and free for its next allocations
        del pending
        with torch.cuda.stream(s):
            torch.cuda._sleep(1_000_000)
        got = call(stream=s)
        pending = junk()  # nor may these take the place of what the call freed while its kernels still wait
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(tensors(got), want))
        del got, pending
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copies = [x.clone() for x in tensors(got)]
    del got
    with torch.cuda.stream(s):
        later = junk()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    del later
