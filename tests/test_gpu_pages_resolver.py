"""The page calls' table as hs_resolve's resident_pages: a step of sequences that grow and branch, of whose tokens
some are on pages, some in hot slots and some on the host, through the resolver, the 4-bit attention and the
backup."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_fp4 as T  # noqa: E402
import test_gpu_pages as G  # noqa: E402
from oracle import fp4_mla as F  # noqa: E402
from oracle import pages as O  # noqa: E402

pytestmark = pytest.mark.gpu

R, MP, PS, P, K, H, CTX = 4, 30, 16, 70, 24, 40, 480


class Server:
    def __init__(self, hs):
        self.hs, self.rng = hs, np.random.default_rng(8)
        # the pages are the pool's first rows, the hot slots' rows stand behind them
        s = self.s = G.Pair(hs, 3, R, MP, P + (R * (H + 1) + PS - 1) // PS, PS)
        s.pool = hs.make_page_pool(s.pools, R, MP, P, PS, 416, s.table, s.refs, s.free, s.count, s.ws, s.ws.numel(), s.err)
        hs.hs_pages_init(s.pool)
        s.orc = O.Pages(R, MP, P, PS, s.orc.pools)
        self.dev, rows = s.pools[0], s.pools[0].shape[0]
        self.host = torch.zeros(2 * R * CTX, 416, dtype=torch.uint8).pin_memory()
        cfg = hs.make_config(R, K, H, 416, 1, PS, CTX, MP)
        self.ws = torch.zeros(hs.hs_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        self.h = hs.hs_create(cfg, [self.host], [self.dev], 2 * R * CTX, rows, self.ws)
        self.hcl = np.arange(R * CTX, dtype=np.int32).reshape(R, CTX)
        self.dbl = P * PS + torch.arange(R * (H + 1), dtype=torch.int32, device="cuda").view(R, H + 1)
        self.tok = torch.full((R, H), -1, dtype=torch.int32, device="cuda")
        self.stamp, self.clock = torch.zeros(R, H, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
        self.rec = {}  # request -> its tokens' rows

    def check_pages(self):
        """The table, counts and stack as the oracle has them (the pool's bytes are the resolver's too)."""
        o, s = self.s.orc, self.s
        assert np.array_equal(s.table.cpu().numpy(), o.table) and np.array_equal(s.refs.cpu().numpy()[:P], o.refs)
        assert s.free.cpu().numpy()[:int(s.count.item())].tolist() == o.free and int(s.err.item()) == 0

    def grow(self, r, k):
        s, start = self.s, len(self.rec.get(r, ()))
        new = T.tokens(self.rng, k)
        self.hs.hs_pages_extend(s.pool, 1, G.d([r]), G.d([start]), G.d([start + k]))
        s.orc.extend([r], [start], [start + k])
        t = np.arange(start, start + k)
        rows = s.orc.table[r, t // PS] * PS + t % PS
        self.hs.hs_fp4_pack_rows(k, T.d(new), 576, G.d(rows), 1.0, self.dev, self.dev.shape[0], s.err)
        rec = F.pack(new, 1.0)
        self.rec[r] = np.concatenate((self.rec[r], rec)) if start else rec
        for i in range(k - 1):  # (the last one goes by hs_backup)
            self.host[self.hcl[r, start + i]] = torch.from_numpy(rec[i])
        self.check_pages()

    def step(self, what):
        """Top-k of every sequence through the resolver, attention over what it names, the newest tokens backed up."""
        hs, rng = self.hs, self.rng
        lens = np.array([len(self.rec.get(r, ())) for r in range(R)], np.int32)
        top = np.full((R, K), -1, np.int32)
        for r in self.rec:
            top[r] = np.concatenate(([lens[r] - 1], rng.permutation(int(lens[r]) - 1)[:K - 1]))
        out, hcl = torch.zeros(R, K, dtype=torch.int32, device="cuda"), G.d(self.hcl)
        before = self.host.clone()
        hs.hs_resolve(self.h, R, G.d(top), G.d(lens), hcl, self.dbl, self.tok, self.stamp, self.clock, self.s.table, out, None)
        hs.hs_backup(self.h, R, G.d(lens), hcl, self.dbl, self.s.table)
        q = T.bf16_bits(rng.standard_normal((R, 16, 576)))
        o, lse, err = T.sparse(hs, q, self.dev, out, 1.0, 1)
        assert err == 0 and hs.hs_get_error(self.h) == 0, what
        for r in self.rec:
            T.check(q[r], self.rec[r][top[r]], 1.0, o[r], lse[r], f"{what}: request {r}")
            before[self.hcl[r, lens[r] - 1]] = torch.from_numpy(self.rec[r][-1])
        assert (o[[r for r in range(R) if r not in self.rec]] == 0).all()
        assert torch.equal(self.host, before), what  # the newest tokens' rows, and no other


def test_sequences_that_branch_through_the_resolver():
    hs = T._gpu()
    v = Server(hs)
    s = v.s
    v.grow(0, 300)
    v.grow(1, 200)
    v.step("two sequences on pages")
    # the middle of request 0 leaves the GPU: its tokens come from the host, through hot slots
    hs.hs_pages_free(s.pool, 1, G.d([0]), G.d([2]), G.d([15]))
    s.orc.release([0], [2], [15])
    v.check_pages()
    for _ in range(2):
        v.step("pages that left")
    # it branches in the middle of a page that is there, and in front of pages that are not
    for child, n in ((2, 300), (3, 245)):
        hs.hs_pages_fork(s.pool, 1, G.d([0]), G.d([child]), G.d([n]))
        s.orc.fork([0], [child], [n])
        v.check_pages()
        v.rec[child] = v.rec[0][:n].copy()
        v.hcl[child, :n] = v.hcl[0, :n]  # the parent's host rows
        v.step(f"a branch at {n}")
    for k in (1, 7, 20):
        for r in (0, 2, 3):
            v.grow(r, k)
        v.step(f"branches {k} tokens on")
    # a sequence ends and the pool is packed: pages move, hot slots and host rows stay
    hs.hs_pages_free(s.pool, 1, G.d([0]))
    s.orc.release([0])
    del v.rec[0]
    hs.hs_pages_compact(s.pool)
    s.orc.compact()
    v.check_pages()
    v.step("the parent is gone")
    v.grow(3, 40)
    v.step("a branch grows on")
    hs.hs_destroy(v.h)
