"""The calls that fill and read the caches as they are used together: a layer over paged caches (pages, norms, rotation, selection,
attention) against the oracle, on streams, in captured graphs, and two calls at once; outputs that a call allocates itself."""
import numpy as np
import pytest
import torch

from oracle import latent4 as o4
from oracle import mla as omla
from oracle import tables as otab
import parity
from test_gpu_cache import SCALE, dev, i32, mla_case, mt, rope_table, status, u32  # noqa: F401

pytestmark = pytest.mark.gpu


def layer(row_bytes, rng, n_pages=60, page=16, H=32):
    from mtp_speculative_decode_gb300 import pipeline
    w = lambda n: dev((1 + 0.2 * rng.normal(size=n)).astype(np.float32))  # noqa: E731
    return pipeline.PagedAttention(3, 320, n_pages, page, dev(rope_table(400, 64)), w(128), dev(rng.normal(size=128).astype(np.float32)),
                                   w(512), H=H, H_I=32, topk=64, max_tokens=300, row_bytes=row_bytes)


def tokens(rng, T, H):
    return dict(q_idx=torch.tensor(rng.normal(size=(T, 32, 128))).to(torch.bfloat16).cuda(),
                k_idx=torch.tensor(rng.normal(size=(T, 128))).to(torch.bfloat16).cuda(),
                w_idx=dev(rng.random((T, 32)).astype(np.float32)),
                q=torch.tensor(rng.normal(size=(T, H, 576)) * 2).to(torch.bfloat16).cuda(),
                kv=torch.tensor(rng.normal(size=(T, 576)) * 3).to(torch.bfloat16).cuda())


def unpacked(latent):
    x = latent.cpu()
    if x.shape[1] == 416:
        return o4.unpack(x.numpy())
    return omla.unpack_fp8_ds_mla(x.numpy()) if x.shape[1] == 656 else x.double().numpy()


@pytest.mark.parametrize("H", [32, 128])
@pytest.mark.parametrize("row_bytes", [416, 656, 1152])
def test_layer_over_paged_caches(mt, row_bytes, H):  # noqa: F811
    """Prompts, then windows, a request that shrinks, one that leaves: tables, slots and positions equal the oracle's, the selection
    attends over what the caches hold."""
    rng = np.random.default_rng(row_bytes + H)
    L = layer(row_bytes, rng, H=H)
    t, free, n_free = L.block_table.cpu().numpy(), L.free_pages.cpu().numpy(), 60
    held = np.zeros(3, np.int64)
    for counts, new in (([100, 7, 0], [100, 7, 0]), ([6, 6, 130], [106, 13, 130]), ([4, 0, 1], [103, 13, 131]), ([6, 6, 6], [109, 19, 137])):
        counts, new = np.array(counts), np.array(new, np.int64)
        off = np.concatenate([[0], np.cumsum(counts)])
        T = int(off[-1])
        x = tokens(rng, T, H)
        plain = x["q"].clone()
        out = L.step(dev(new), u32(off), **x)
        t, held, n_free, st = otab.grow(t, 16, new, free, n_free, held)
        slots, pos, _, _ = otab.slot_map(t, 16, off, new, T)
        assert st == 0 and L.status.item() == 0 and L.n_free.item() == n_free
        assert np.array_equal(L.block_table.cpu().numpy(), t) and np.array_equal(L.lengths.cpu().numpy(), held)
        assert np.array_equal(L.slots[:T].cpu().numpy(), slots) and np.array_equal(L.positions[:T].cpu().numpy(), pos)
        assert torch.equal(x["q"][:, :, :512], plain[:, :, :512]) and not torch.equal(x["q"][:, :, 512:], plain[:, :, 512:])
        # the step's rows are in the caches: the norm of the latent's float64 values, within the format's steps
        rows = unpacked(L.latent)
        kv = x["kv"].double().cpu().numpy()[:, :512]
        want = kv / np.sqrt((kv * kv).mean(1, keepdims=True) + 1e-6) * L.latent_weight.double().cpu().numpy()
        blocks = np.abs(want).reshape(T, -1, 16).max(2).repeat(16, 1)
        step = {416: blocks / 5.5, 656: np.abs(want) / 16 + np.abs(want).max(1, keepdims=True) / 448 / 512,
                1152: np.abs(want) / 256}[row_bytes]
        assert (np.abs(rows[slots][:, :512] - want) <= step * 1.001 + 1e-6).all()
        idx = L.topk_idx[:T].cpu().numpy()
        req = np.repeat(np.arange(3), counts)
        for r in list(range(0, T, 17)) + [T - 1]:
            sel = idx[r][idx[r] >= 0]
            assert len(sel) == min(64, pos[r] + 1) and sel.max() <= pos[r]
            at = np.array([t[req[r], s // 16] * 16 + s % 16 for s in sel])
            o, _ = omla.sparse_mla(x["q"][r:r + 1].cpu(), rows[at], [0], [0], np.arange(len(at))[None], SCALE)[0]
            parity.check_attention_row(out[r].float().cpu().numpy(), o, parity.ATT_TOL_BF16)
    keep = np.array([50, 0, 137], np.int64)
    L.release(dev(keep))
    t, free, n_free, _ = otab.release(t, 16, held, free, n_free, keep)
    assert np.array_equal(L.block_table.cpu().numpy(), t) and L.n_free.item() == n_free
    assert np.array_equal(L.free_pages.cpu().numpy(), free) and np.array_equal(L.lengths.cpu().numpy(), np.minimum(held, keep))
    L.release()
    assert L.n_free.item() == 60 and sorted(L.free_pages.tolist()) == list(range(60)) and (L.block_table == -1).all()


def test_layer_without_pages(mt):  # noqa: F811
    """A request that gets no pages: flagged, nothing of it is written, the others run."""
    rng = np.random.default_rng(1)
    L = layer(416, rng, n_pages=8)
    x = tokens(rng, 150, 32)
    out = L.step(dev(np.array([100, 50, 0], np.int64)), u32([0, 100, 150, 150]), **x)
    assert L.status.item() == 32 | 8 | 2 and L.lengths.tolist() == [100, 0, 0] and (L.block_table[1:] == -1).all()
    assert (L.slots[100:150] == -1).all() and torch.isfinite(out[:100].float()).all()


@pytest.mark.parametrize("page", [None, 64])
def test_decode_step_over_4_bit_caches(mt, page):  # noqa: F811
    """The decode step's latent caches in 4 bits, contiguous and paged, against the oracle over the unpacked rows."""
    import dataclasses
    from mtp_speculative_decode_gb300 import pipeline, workloads
    w = workloads.build(dataclasses.replace(workloads.SPECS["verify"], B=2, lengths=[5000, 3000]))
    g = pipeline.DecodeStep(w, "cuda:0", latent_fp4=True, page_size=page)
    g.step()
    torch.cuda.synchronize()
    assert g.status.item() == 0 and g.latent.shape[1] == 416
    idx, per = g.topk_idx.cpu().numpy(), g.R // g.B
    for r in (0, per - 1, per, g.R - 1):
        b, sel = r // per, idx[r][idx[r] >= 0]
        if page:
            at = g.block_table_host[b, sel // page].astype(np.int64) * page + sel % page
        else:
            at = int(w.cache_start[b]) + sel.astype(np.int64)
        rows = o4.unpack(g.latent[torch.from_numpy(at).cuda()].cpu().numpy())
        o, lse = omla.sparse_mla(g.q_mla[r:r + 1].cpu(), rows, [0], [0], np.arange(len(at))[None], workloads.SOFTMAX_SCALE)[0]
        parity.check_attention_row(g.out[r].float().cpu().numpy(), o, parity.ATT_TOL_BF16)
        assert np.abs(g.lse[r].cpu().numpy() - lse).max() <= 2e-2
    with pytest.raises(ValueError):
        pipeline.DecodeStep(w, "cuda:0", latent_fp4=True, latent_fp8=True)


def calls(m):
    """name -> (call(stream) -> outputs): every call on inputs of its own."""
    rng = np.random.default_rng(4)
    g = torch.Generator(device="cuda").manual_seed(4)
    T, H = 700, 8
    q = torch.randn(T, H, 128, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn(T, 576, generator=g, device="cuda").to(torch.bfloat16)
    cs, pos = dev(rope_table(500, 64)), torch.randint(0, 500, (T,), generator=g, device="cuda")
    new = torch.randint(0, 4000, (90,), generator=g, device="cuda")
    off = u32(np.concatenate([[0], np.cumsum(new.cpu().numpy())]))
    table = torch.zeros(90, 300, dtype=torch.int32, device="cuda")
    free, n_free = torch.randperm(30000, generator=g, device="cuda").to(torch.int32), i32([30000])
    slots, n_out = torch.zeros(int(new.sum()), dtype=torch.int64, device="cuda"), i32([0])
    mq, rows, caps, start, mpos, idx = mla_case(rng, 3, 2, 128, 1500, [4000, 2500, 9])
    mla = (mq.cuda(), dev(rows), dev(start), u32([0, 2, 4, 6]), dev(mpos), dev(idx), SCALE)
    few = (mla[0][:, :48].contiguous(),) + mla[1:]

    def grow(s):
        lengths = m.block_table_grow(table, 16, new, free, n_free, n_free_out=n_out, token_offsets=off, slots=slots, stream=s)
        return [lengths, table, slots, n_out]

    return {"norm_rope": lambda s: list(m.norm_rope(pos, cs, q=q, k=kv, q_norm="rms", k_norm="layer", stream=s)),
            "pack_latent_fp4": lambda s: [m.pack_latent_fp4(kv, stream=s)], "block_table_grow": grow,
            "mla": lambda s: [m.sparse_mla_decode(*mla, stream=s)], "mla_few_heads": lambda s: [m.sparse_mla_decode(*few, stream=s)]}


NAMES = ["norm_rope", "pack_latent_fp4", "block_table_grow", "mla", "mla_few_heads"]


@pytest.mark.parametrize("name", NAMES)
def test_streams_and_graphs(mt, name):  # noqa: F811
    """On a side stream (object and raw handle), captured and replayed, and twice from two graphs at once: the same bits."""
    call = calls(mt)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = call(s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(None)
        graphs.append((g, out))
    other = torch.cuda.Stream()
    for _ in range(3):
        for _, out in graphs:
            for x in out:
                x.zero_()
        torch.cuda.synchronize()
        graphs[0][0].replay()
        # (the two graphs of the tables share their outputs: one after the other)
        with torch.cuda.stream(torch.cuda.current_stream() if name == "block_table_grow" else other):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_attention_calls_at_once(mt):  # noqa: F811
    """Split calls on two streams at the same time, without a workspace given: neither sees the other's partials."""
    rng = np.random.default_rng(12)
    sets = []
    for H in (128, 64):
        q, rows, caps, start, pos, idx = mla_case(rng, 2, 1, H, 2000, [6000, 3000])
        sets.append((q.cuda(), dev(rows), dev(start), u32([0, 1, 2]), dev(pos), dev(idx), SCALE))
    want = [mt.sparse_mla_decode(*a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [mt.sparse_mla_decode(*a, stream=s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
