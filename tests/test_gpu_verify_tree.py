"""shortconv_kv_verify_tree: a chain gives the bits of shortconv_kv_verify; a tree gives, token by
token, the bits of a chain along that token's path; refusals of the device indices; and a serving
program's steps in a row (verify, attention, commit, scores, eviction, decode)."""
import numpy as np
import pytest
import torch

import causal_short_convolution_amd as sc
from cache_problem import DEV, check_rows
import cache_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Step:
    def __init__(self, seed, dtype=torch.bfloat16, H=2, D=64, W=4, drafts=(5, 0, 9), chain=False,
                 pad=0, behind=0, spare=6):
        g = np.random.default_rng(seed)
        tg = torch.Generator().manual_seed(seed)
        self.N, self.H, self.D, self.W, self.dt = len(drafts), H, D, W, dtype
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.T = int(self.cu[-1]) + behind
        self.M = max(max(drafts), 1)
        self.parents = np.full(self.T, -1, np.int32)
        for s, n in enumerate(drafts):
            for i in range(1, n):
                self.parents[self.cu[s] + i] = (i - 1 if chain else
                                                -1 if g.random() < 0.1 else g.integers(max(0, i - 4), i))

        def rows():
            base = torch.randn((self.T, H * D + pad), generator=tg).to(dtype).to(DEV)
            return base[:, :H * D].view(self.T, H, D)

        r = lambda *shape: torch.randn(shape, generator=tg).to(DEV)
        self.k, self.v = rows(), rows()
        self.params = [r(W, H, D) * W ** -0.5, r(W, H, D) * W ** -0.5, 1 + 0.1 * r(D),
                       1 + 0.1 * r(D)]
        self.states = ([r(self.N + 2, W - 1, H, D).to(dtype) for _ in range(2)] if W > 1 else
                       [None, None])
        self.sidx = torch.from_numpy(g.permutation(self.N + 2)[:self.N].astype(np.int32)).to(DEV)
        self.slots = self.T + spare
        self.slot = torch.from_numpy(g.permutation(self.slots)[:self.T].astype(np.int64)).to(DEV)

    def buffers(self, mx=False, M=None):
        M = self.M if M is None else M
        if mx:
            kv = [torch.full((self.slots, self.H, self.D), 0x55, dtype=torch.uint8, device=DEV)
                  for _ in range(2)]
            kv += [torch.full((self.slots, self.H, self.D // 32), 0x55, dtype=torch.uint8,
                              device=DEV) for _ in range(2)]
        else:
            kv = [torch.full((self.slots, self.H, self.D), 7.0, dtype=self.dt, device=DEV)
                  for _ in range(2)]
        snap = ([torch.full((self.N, M, self.W - 1, self.H, self.D), 5.0, dtype=self.dt, device=DEV)
                 for _ in range(2)] if self.W > 1 else [None, None])
        return kv, snap

    def tree(self, kv, snap, mask=None, parents=None, mx=False, stream=None):
        f = sc.shortconv_kv_verify_tree_mxfp8 if mx else sc.shortconv_kv_verify_tree
        f(self.k, self.v, torch.from_numpy(self.cu).to(DEV),
          torch.from_numpy(self.parents if parents is None else parents).to(DEV), *self.params,
          1e-6, *self.states, self.sidx, *snap, self.slot, *kv, mask=mask, stream=stream)
        torch.cuda.synchronize()

    def path(self, s, i):
        out = []
        while i >= 0:
            out.append(i)
            p = int(self.parents[self.cu[s] + i])
            i = p if 0 <= p < i else -1
        return out[::-1]

    def along_paths(self, mx):
        """The chain entry points, run on every token's path as a sequence of its own; the rows of
        the paths' last tokens are kept."""
        tokens, owner, lens = [], [], []
        for s in range(self.N):
            for i in range(int(self.cu[s + 1] - self.cu[s])):
                path = self.path(s, i)
                tokens += [int(self.cu[s]) + j for j in path]
                owner.append(s)
                lens.append(len(path))
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
        at = torch.tensor(tokens, device=DEV)
        slot = torch.full((len(tokens),), -1, dtype=torch.int64, device=DEV)
        slot[(cu[1:] - 1).long()] = self.slot[:len(lens)]
        k, v = self.k[at].contiguous(), self.v[at].contiguous()
        states = [None if t is None else t[self.sidx.long()[owner]].contiguous()
                  for t in self.states]
        kv, _ = self.buffers(mx)
        f = sc.shortconv_kv_prefill_mxfp8 if mx else sc.shortconv_kv_prefill
        f(k, v, cu, *self.params, 1e-6, *states, None, None, slot, *kv)
        torch.cuda.synchronize()
        return kv, states  # the prefill leaves each path's new state in the pool


def bits(t):
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def same(a, b):
    return all(x is None and y is None or torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (3, 256)])
@pytest.mark.parametrize("W", [1, 2, 4, 8])
def test_chain_equals_verify(dtype, H, D, W):
    st = Step(W, dtype, H, D, W, drafts=(5, 0, 1, 9, 33), chain=True, pad=16)
    kv, snap = st.buffers()
    st.tree(kv, snap)
    kv2, snap2 = st.buffers()
    sc.shortconv_kv_verify(st.k, st.v, torch.from_numpy(st.cu).to(DEV), *st.params, 1e-6,
                           *st.states, st.sidx, *snap2, st.slot, *kv2)
    torch.cuda.synchronize()
    assert same(kv, kv2) and same(snap, snap2)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (3, 256)])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
def test_tree_equals_chains_along_the_paths(mx, dtype, H, D, W):
    st = Step(10 + W, dtype, H, D, W, drafts=(5, 0, 1, 70, 9))
    kv, snap = st.buffers(mx)
    mask = torch.full((st.T, 2), -1, dtype=torch.int64, device=DEV)
    st.tree(kv, snap, mask, mx=mx)
    kv2, states = st.along_paths(mx)
    assert same(kv, kv2)
    if W > 1:
        t = 0
        for s in range(st.N):
            n = int(st.cu[s + 1] - st.cu[s])
            for snaps, new in zip(snap, states):
                assert torch.equal(bits(snaps[s, :n]), bits(new[t:t + n]))
                assert bool((snaps[s, n:] == 5.0).all())
            t += n
    got = mask.cpu().numpy().view(np.uint64)
    for s in range(st.N):
        for i in range(int(st.cu[s + 1] - st.cu[s])):
            want = np.zeros(2, np.uint64)
            for j in st.path(s, i):
                want[j // 64] |= np.uint64(1 << (j % 64))
            assert (got[st.cu[s] + i] == want).all()


def test_bad_parents_make_roots_and_rows_behind_stay():
    st = Step(30, drafts=(6, 4), behind=3)
    bad = st.parents.copy()
    bad[[1, 3, 7]] = [1, 5, -9]      # itself, a later token, below -1
    bad[9] = 2 ** 31 - 1
    st.parents[[1, 3, 7, 9]] = -1    # what they stand for
    want = st.buffers()
    st.tree(*want)
    got = st.buffers()
    mask = torch.full((st.T, 1), -3, dtype=torch.int64, device=DEV)
    st.tree(*got, mask=mask, parents=bad)
    assert same(got[0], want[0]) and same(got[1], want[1])
    assert bool((mask[-3:] == -3).all())
    untouched = torch.ones(st.slots, dtype=torch.bool, device=DEV)
    untouched[st.slot[:10]] = False
    assert all(bool((t[untouched] == 7.0).all()) for t in got[0])


def test_no_state_few_snapshots_few_words_and_skipped_slots():
    st = Step(31, W=3, drafts=(70, 3))
    st.sidx[1] = 99                      # outside the pool: zeros
    st.slot[::5] = -1
    kv, snap = st.buffers(M=4)
    mask = torch.zeros((st.T, 1), dtype=torch.int64, device=DEV)
    st.tree(kv, snap, mask=mask)
    zero = Step(31, W=3, drafts=(70, 3))
    zero.slot[::5] = -1
    for t in zero.states:
        t[zero.sidx[1].long()] = 0
    kv2, snap2 = zero.buffers()
    full = torch.zeros((st.T, 2), dtype=torch.int64, device=DEV)
    zero.tree(kv2, snap2, mask=full)
    assert same(kv, kv2) and all(torch.equal(a, b[:, :4]) for a, b in zip(snap, snap2))
    assert torch.equal(mask[:, 0], full[:, 0])
    none = Step(31, W=3, drafts=(70, 3))
    none.states = [None, None]
    kv3, snap3 = none.buffers()
    none.tree(kv3, snap3)
    for t in zero.states:
        t.zero_()
    kv4, snap4 = zero.buffers()
    none.slot[::5] = -1
    kv3, snap3 = none.buffers()
    none.tree(kv3, snap3)
    zero.tree(kv4, snap4)
    assert same(kv3, kv4) and same(snap3, snap4)


def test_large_batch_and_side_stream():
    st = Step(32, H=4, D=128, drafts=[1 + i % 12 for i in range(150)])
    want = st.buffers()
    st.tree(*want)
    kv2, _ = st.along_paths(False)
    assert same(want[0], kv2)
    side = torch.cuda.Stream()
    got = st.buffers()
    torch.cuda.synchronize()
    st.tree(*got, stream=side)
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_serving_steps_in_a_row():
    """Prompt prefill, a drafted tree verified and attended, the longest accepted path committed,
    weights accumulated, the cache cut to a budget, and a decode step over what is left."""
    H, G, D, W, bs, N = 2, 4, 64, 4, 16, 2
    lens, drafts = [90, 37], [6, 6]
    g = torch.Generator(device=DEV).manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    bf = torch.bfloat16
    params = [r(W, H, D) / 2, r(W, H, D) / 2, 1 + 0.1 * r(D), 1 + 0.1 * r(D)]
    MB = 8
    table = torch.randperm(20, generator=g, device=DEV)[:N * MB].view(N, MB).to(torch.int32)
    kc, vc = (torch.full((20 * bs, H, D), float("nan"), dtype=bf, device=DEV) for _ in range(2))
    state = [torch.zeros((N, W - 1, H, D), dtype=bf, device=DEV) for _ in range(2)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    slots = lambda s, a, b: [int(table[s, p // bs]) * bs + p % bs for p in range(a, b)]

    cu = i32([0, lens[0], sum(lens)])
    k, v = r(sum(lens), H, D).to(bf), r(sum(lens), H, D).to(bf)
    where = torch.tensor(slots(0, 0, lens[0]) + slots(1, 0, lens[1]), device=DEV)
    sc.shortconv_kv_prefill(k, v, cu, *params, 1e-6, *state, None, i32([0, 0]).to(torch.uint8),
                            where, kc, vc)

    cu = i32([0, 6, 12])
    parents = i32([-1, 0, 0, 1, 3, 2] * 2)
    k, v = r(12, H, D).to(bf), r(12, H, D).to(bf)
    snap = [torch.zeros((N, 6, W - 1, H, D), dtype=bf, device=DEV) for _ in range(2)]
    mask = torch.zeros((12, 1), dtype=torch.int64, device=DEV)
    where = torch.tensor(slots(0, 90, 96) + slots(1, 37, 43), device=DEV)
    sc.shortconv_kv_verify_tree(k, v, cu, parents, *params, 1e-6, *state, None, *snap, where, kc,
                                vc, mask=mask)
    assert mask[:6, 0].tolist() == [1, 3, 5, 11, 27, 37]
    q = r(12, H * G, D).to(bf)
    out = torch.empty_like(q)
    lse = torch.empty((12, H * G), device=DEV)
    ctx = i32(lens)
    sc.shortconv_tree_attention(q, cu, ctx, table, bs, kc, vc, out, mask=mask, lse=lse)
    torch.cuda.synchronize()
    host = lambda t: t.cpu().numpy()
    kvals, vvals = host(kc.double()), host(vc.double())
    want = ref.attention(host(q.double()), host(cu), host(ctx), host(table), bs, kvals, vvals,
                         20 * bs, D ** -0.5, bf, mask=host(mask).view(np.uint64))
    check_rows(want, out, lse)

    # the verifier accepts the path 0-1-3-4 of the first tree and 0-2 of the second
    sc.shortconv_state_commit(*snap, cu, 12, i32([5, 3]), *state, None, width=W, num_heads=H,
                              head_dim=D)
    torch.cuda.synchronize()
    assert torch.equal(state[0][0], k[[1, 3, 4]]) and torch.equal(state[1][1][1:], v[[6, 8]])

    cap = MB * bs
    weight = torch.zeros((N, H, cap), device=DEV)
    sc.shortconv_cache_scores(q, lse, cu, ctx, table, bs, kc, None, weight, mask=mask)
    positions = torch.arange(cap, dtype=torch.int32, device=DEV).expand(N, H, cap).contiguous()
    length = i32([96, 43])
    seen = length.clone()
    before = (kc.clone(), vc.clone(), weight.clone())
    sc.shortconv_cache_evict(weight, positions, length, seen, 40, table, bs, kc, vc, weight,
                             positions, length, sinks=4, recent=8)
    torch.cuda.synchronize()
    assert length.tolist() == [40, 40]
    kvals = host(kc.double())
    for s in range(N):
        n = [96, 43][s]
        for h in range(H):
            kept = positions[s, h, :40].tolist()
            assert len(set(kept)) == 40 and set(range(4)) | set(range(n - 8, n)) <= set(kept)
            dropped = sorted(set(range(4, n - 8)) - set(kept))
            inner = [p for p in kept if 4 <= p < n - 8]
            w = before[2][s, h]
            assert float(w[inner].min()) >= float(w[dropped].max())
            for j, p in enumerate(kept):
                a, b = slots(s, j, j + 1)[0], slots(s, p, p + 1)[0]
                assert torch.equal(kc[a, h], before[0][b, h]) and torch.equal(vc[a, h], before[1][b, h])

    # decode over the 40 kept entries: the new row goes to position 40
    k1, v1 = r(N, H, D).to(bf), r(N, H, D).to(bf)
    where = torch.tensor(slots(0, 40, 41) + slots(1, 40, 41), device=DEV)
    sc.shortconv_kv_decode(k1, v1, *params, 1e-6, *state, None, where, kc, vc)
    q = r(N, H * G, D).to(bf)
    out = torch.empty_like(q)
    cu = i32([0, 1, 2])
    sc.shortconv_tree_attention(q, cu, length, table, bs, kc, vc, out)
    torch.cuda.synchronize()
    want = ref.attention(host(q.double()), host(cu), host(length), host(table), bs,
                         host(kc.double()), host(vc.double()), 20 * bs, D ** -0.5, bf)
    check_rows(want, out, None)
