"""The windowed calls as a serving loop uses them together: prompts prefilled in
chunks, then decoding, with rotary positions on every token, the pages behind
the window freed and handed to other sequences; against dense attention in 64
bits over the rows that were actually written."""
import numpy as np
import pytest

import workloads as wl
from paged_inputs import to_f64
from window_reference import EPS, attend, rotate, seen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")


class Server:
    """One attention layer over a pool too small to hold the whole contexts."""

    def __init__(self, seed, hq, hkv, d, dtype, window, sinks, blocks, interleaved, sections):
        self.rng = wl.rng_for(seed)
        self.hq, self.hkv, self.d, self.dtype = hq, hkv, d, dtype
        self.window, self.sinks, self.scale = window, sinks, 1.0 / np.sqrt(d)
        self.alloc = pk.BlockAllocator(blocks)
        self.blocks = blocks
        nan = torch.full((blocks, hkv, 16, d), float("nan"), dtype=gh.tdtype(dtype), device="cuda")
        self.kc, self.vc = nan, nan.clone()
        pairs = sum(sections)
        self.freq = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
        self.axes = np.repeat(np.arange(len(sections)), sections)
        self.interleaved = interleaved
        self.rope = pk.Rope(self.freq, self.axes, interleaved=interleaved)
        self.kept = {}  # sequence -> list of (k row, v row) in 64 bits, as cached

    def project(self, T):
        x = wl.draw_values(self.rng, (T, self.hq + 2 * self.hkv, self.d), self.dtype)
        return x, gh.to_dev(x, self.dtype)

    def positions(self, at):
        """[axes][T]: the time axis follows the token, the others walk a grid."""
        at = np.asarray(at)
        return np.stack([at if a == 0 else (at * (a + 2)) % 37 for a in range(self.axes.max() + 1)]).astype(np.int32)

    def rope_and_cache(self, bits, x, pos, slots, seqs):
        hq, hkv = self.hq, self.hkv
        q = torch.empty((x.shape[0], hq, self.d), dtype=x.dtype, device="cuda")
        pk.rope_and_cache(q, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], self.kc, self.vc,
                          gh.ints(slots, torch.int64), gh.ints(pos), self.rope)
        # the rows as they are in the cache (their own rounding is tested apart)
        k = self.kc.transpose(1, 2).reshape(-1, hkv, self.d)[torch.from_numpy(slots).cuda()]
        want = rotate(to_f64(bits, self.dtype), pos, self.freq, self.axes, self.interleaved)
        k = gh.to_f64(k)
        # half a step of values below 8
        assert np.abs(k - want[:, hq:hq + hkv]).max() <= EPS[self.dtype] * 4
        for t, s in enumerate(seqs):
            self.kept.setdefault(s, []).append((k[t], to_f64(bits[t, hq + hkv:], self.dtype)))
        return q

    def check(self, out, q, rows, seqs):
        """rows[i] query rows per sequence, at the end of its context."""
        half, r0 = EPS[self.dtype] / 2, 0
        G = self.hq // self.hkv
        g, qf = gh.to_f64(out), gh.to_f64(q)
        for n, s in zip(rows, seqs):
            K = np.stack([k for k, _ in self.kept[s]])
            V = np.stack([v for _, v in self.kept[s]])
            L = len(K)
            mask = seen(np.arange(L - n, L), np.arange(L), self.window, self.sinks)
            for h in range(self.hkv):
                hs = slice(h * G, (h + 1) * G)
                ref, mean = attend(qf[r0:r0 + n, hs], K[:, h], V[:, h], mask, self.scale)
                tol = (half + 2.0 ** -12) * mean + half * np.abs(ref) + 1e-7
                assert np.all(np.abs(g[r0:r0 + n, hs] - ref) <= tol)
            r0 += n

    def tables(self, seqs, width):
        t, lens = self.alloc.build_tables(seqs, width)
        return gh.ints(t), gh.ints(lens), t, lens


@pytest.mark.parametrize("hq,hkv,d,dtype,window,sinks,interleaved,sections", [
    (8, 2, 128, wl.BF16, 100, 4, False, (16, 24, 24)),
    (4, 4, 64, wl.F16, 33, 20, True, (8, 8)),
    (12, 1, 64, wl.BF16, 64, 0, False, (24,)),
])
def test_chunked_prompts_then_decoding_in_a_small_pool(hq, hkv, d, dtype, window, sinks, interleaved,
                                                       sections):
    prompts, width = [230, 75, 140], 32
    # each sequence at its widest: the sinks, the window, a chunk and its ends
    blocks = len(prompts) * (-(-sinks // 16) + (window + 64) // 16 + 4)
    assert blocks < sum(-(-(n + 40) // 16) for n in prompts) or window > 90
    srv = Server(7, hq, hkv, d, dtype, window, sinks, blocks, interleaved, sections)
    seqs = list(range(len(prompts)))
    done = [0] * len(prompts)
    for s in seqs:
        srv.alloc.add_seq(s, 0)
    freed = 0
    # chunks of the prompts, ragged, until every prompt is in
    while any(done[s] < prompts[s] for s in seqs):
        live = [s for s in seqs if done[s] < prompts[s]]
        n = [min(int(srv.rng.integers(1, 64)), prompts[s] - done[s]) for s in live]
        slots = np.concatenate([[srv.alloc.append_slot(s)[0] for _ in range(m)] for s, m in zip(live, n)])
        at = np.concatenate([np.arange(done[s], done[s] + m) for s, m in zip(live, n)])
        bits, x = srv.project(len(at))
        q = srv.rope_and_cache(bits, x, srv.positions(at), slots.astype(np.int64), np.repeat(live, n))
        tbl, lens, t, _ = srv.tables(live, width)
        start = gh.ints(np.concatenate([[0], np.cumsum(n)]))
        out = torch.full_like(q, float("nan"))
        size = pk.prefill_window_workspace_size(len(live), len(at), max(n), hq, hkv, d, width, window, sinks)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        pk.prefill_window(out, q, srv.kc, srv.vc, tbl, lens, start, max(n), hkv, srv.scale, window, sinks,
                          workspace=ws)
        assert pk.get_error() == (0, 0)
        srv.check(out, q, n, live)
        for s, m in zip(live, n):
            done[s] += m
            freed += srv.alloc.trim_window(s, done[s], window, sinks)
    # decoding: the write inside the call on even steps, before it on odd ones
    for step in range(24):
        slots, pairs = srv.alloc.append_slots(seqs)
        assert not len(pairs)
        at = np.array([srv.alloc.num_tokens(s) - 1 for s in seqs])
        bits, x = srv.project(len(seqs))
        q = srv.rope_and_cache(bits, x, srv.positions(at), slots, seqs)
        tbl, lens, t, L = srv.tables(seqs, width)
        out = torch.full_like(q, float("nan"))
        if step % 2:
            pk.decode_window(out, q, srv.kc, srv.vc, tbl, lens, hkv, srv.scale, window, sinks)
        else:
            k = srv.kc.transpose(1, 2).reshape(-1, hkv, d)[torch.from_numpy(slots).cuda()].contiguous()
            v = x[:, hq + hkv:].contiguous()
            pk.decode_append_window(out, q, k, v, srv.kc, srv.vc, tbl, lens, hkv, srv.scale, window, sinks)
        assert pk.get_error() == (0, 0)
        srv.check(out, q, [1] * len(seqs), seqs)
        for s in seqs:
            freed += srv.alloc.trim_window(s, srv.alloc.num_tokens(s), window, sinks)
    assert freed > 0
    for s in seqs:
        srv.alloc.free_seq(s)
    assert srv.alloc.stats()["free_blocks"] == blocks


def test_one_captured_step_serves_growing_contexts():
    """The plan depends on the table's width only: lengths, tables and rows may
    change between replays of one captured step."""
    hq, hkv, d, window, sinks, S, width = 16, 4, 128, 200, 4, 5, 64
    rng = wl.rng_for(11)
    rope = pk.Rope(10000.0 ** (-np.arange(64) / 64), [0] * 32 + [1] * 32)
    blocks = S * width
    kc = torch.randn(blocks, hkv, 16, d, device="cuda").bfloat16()
    vc = torch.randn(blocks, hkv, 16, d, device="cuda").bfloat16()
    x = torch.zeros((S, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q, out = torch.empty((S, hq, d), dtype=x.dtype, device="cuda"), torch.empty((S, hq, d), dtype=x.dtype, device="cuda")
    slots = torch.zeros(S, dtype=torch.int64, device="cuda")
    pos = torch.zeros((2, S), dtype=torch.int32, device="cuda")
    lens = torch.ones(S, dtype=torch.int32, device="cuda")
    tbl = torch.from_numpy(rng.permutation(blocks).astype(np.int32).reshape(S, width)).cuda()

    def step():
        pk.rope_and_cache(q, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, slots, pos, rope)
        pk.decode_window(out, q, kc, vc, tbl, lens, hkv, 0.1, window, sinks)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the calls' first use on these shapes
        step()
    for L in (1, 17, 200, 203, 1000, 1024):
        n = np.array([L, max(1, L - 1), (L + 1) // 2, 1, L])
        t = tbl.cpu().numpy()
        lens.copy_(gh.ints(n))
        slots.copy_(gh.ints(t[np.arange(S), (n - 1) // 16].astype(np.int64) * 16 + (n - 1) % 16, torch.int64))
        pos.copy_(gh.ints(np.stack([n - 1, (n * 7) % 50])))
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got, k1 = out.clone(), kc.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(k1, kc)
        assert pk.get_error() == (0, 0)
        K = kc.double()[tbl.long()].transpose(2, 3).reshape(S, width * 16, hkv, d)
        V = vc.double()[tbl.long()].transpose(2, 3).reshape(S, width * 16, hkv, d)
        for s in range(S):
            p = int(n[s]) - 1
            keys = np.nonzero(seen([p], np.arange(p + 1), window, sinks)[0])[0]
            for h in range(hkv):
                ref, mean = attend(gh.to_f64(q)[s:s + 1, 4 * h:4 * h + 4], K[s, keys, h].cpu().numpy(),
                                   V[s, keys, h].cpu().numpy(), np.ones((1, len(keys)), bool), 0.1)
                half = 2.0 ** -8
                tol = (half + 2.0 ** -12) * mean + half * np.abs(ref) + 1e-7
                assert np.all(np.abs(gh.to_f64(got)[s:s + 1, 4 * h:4 * h + 4] - ref) <= tol)


def test_two_streams_with_their_own_workspaces():
    """Overlapping calls that share nothing but the pool give the same bits."""
    rng = wl.rng_for(13)
    hq, hkv, d, S, width, window = 32, 8, 128, 40, 300, 4000
    kc = torch.randn(3000, hkv, 16, d, device="cuda").bfloat16()
    vc = torch.randn(3000, hkv, 16, d, device="cuda").bfloat16()
    jobs = []
    for i in range(2):
        tbl = torch.from_numpy(rng.integers(0, 3000, size=(S, width)).astype(np.int32)).cuda()
        lens = torch.from_numpy(rng.integers(1, width * 16, size=S).astype(np.int32)).cuda()
        q = torch.randn(S, hq, d, device="cuda").bfloat16()
        n = pk.decode_window_workspace_size(S, hq, hkv, d, width, window, 4)
        assert n > 0
        jobs.append([q, tbl, lens, torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q),
                     torch.cuda.Stream()])

    def run(job, stream):
        q, tbl, lens, ws, out, _ = job
        pk.decode_window(out, q, kc, vc, tbl, lens, hkv, 0.09, window, 4, workspace=ws, stream=stream)

    want = []
    for job in jobs:
        run(job, None)
        torch.cuda.synchronize()
        want.append(job[4].clone())
        job[4].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for job in jobs:
            run(job, job[5])
    torch.cuda.synchronize()
    for job, w in zip(jobs, want):
        assert torch.equal(job[4], w)
