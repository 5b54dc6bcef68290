"""The latent cache's operators, and the norm and rotation ahead of the append, as a
program uses them: in steps one after the other, captured and replayed, on other
streams, at the far end of large pools; and what the binding refuses."""
import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

import lat_reference as ref
from test_gpu_latent import close, dev, exp_case, exp_check, exp_run, f64, lat_case, lat_check, lat_run

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()


@pytest.fixture(autouse=True)
def _clean():
    yield
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0


# ------------------------------------------------------------ a serving loop
class Loop:
    """Requests of a model layer with a latent cache: its step builds the step's
    buffers, appends, and attends in both forms."""

    def __init__(self, R, cols, nb, cap, H, rows, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.R, self.cap, self.H, self.nb = g, R, cap, H, nb
        i32 = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
        self.table, self.lens, self.new, self.keep = i32(R, cols), i32(R), i32(R), i32(R)
        self.qsl, self.slots = i32(R + 1), torch.zeros(cap, dtype=torch.int64, device="cuda")
        self.free, self.nfree, self.refused = torch.arange(nb, dtype=I32, device="cuda"), i32(1) + nb, i32(1)
        self.pool = torch.full((nb, 16, 576), float("nan"), dtype=BF, device="cuda")
        self.w = (torch.randn(H, 256, 512, generator=g) / 20).to(BF).cuda()
        self.weight = (1 + 0.2 * torch.randn(512, generator=g)).to(BF).cuda()
        self.cs = torch.from_numpy(ref.table(cols * 16, 64)).cuda()
        self.kv_new, self.q = (torch.zeros(cap, *s, dtype=BF, device="cuda") for s in ((576,), (H, 192)))
        self.pos, self.ksl = torch.zeros(cap, dtype=torch.int64, device="cuda"), i32(R + 1)
        self.q_abs = torch.zeros(cap, H, 576, dtype=BF, device="cuda")
        self.kv, self.kr = torch.zeros(rows, H, 256, dtype=BF, device="cuda"), torch.zeros(rows, 64, dtype=BF, device="cuda")
        self.out, self.lat = (torch.zeros(cap, H, d, dtype=BF, device="cuda") for d in (128, 512))
        self.ws = pkv.LatentWorkspace()
        self.scale = 192 ** -0.5

    def inputs(self, new):
        self.new.copy_(torch.tensor(new, dtype=I32))
        self.kv_new.copy_(torch.randn(self.cap, 576, generator=self.g) * 3)
        self.q.copy_(torch.randn(self.cap, self.H, 192, generator=self.g))
        self.out.fill_(7.0), self.lat.fill_(7.0)

    def step(self):
        pkv.pkv_build_step(self.lens, self.new, self.free, self.nfree, self.table, self.lens, self.qsl, self.slots,
                           num_refused=self.refused)
        # the tokens' positions and the running sum of the lengths, as a program has them
        t = torch.arange(self.cap, device="cuda")
        r = torch.searchsorted(self.qsl, t, right=True, out_int32=True).long().clamp_(1, self.R) - 1
        torch.add(self.lens[r] - self.qsl[r + 1], t, out=self.pos)
        self.ksl[1:] = torch.cumsum(self.lens, 0)
        pkv.pkv_append_latent(self.kv_new, self.pos, self.cs, self.slots, self.pool, weight=self.weight,
                              q_rope=self.q[:, :, 128:])
        self.q_abs[..., :512] = torch.einsum("thd,hdc->thc", self.q[..., :128].float(), self.w[:, :128].float())
        self.q_abs[..., 512:] = self.q[..., 128:]
        pkv.pkv_attention_latent(self.q_abs, self.pool, self.table, self.lens, self.qsl, self.scale, out=self.lat,
                                 workspace=self.ws)
        pkv.pkv_expand_latent(self.pool, self.w, self.table, self.lens, self.ksl, self.kv, self.kr)
        pkv.pkv_attention_expanded(self.q, self.kv, self.kr, self.lens, self.qsl, self.ksl, self.scale, out=self.out,
                                   workspace=self.ws)

    def check(self, before):
        lens, qsl, tab = (x.cpu().numpy() for x in (self.lens, self.qsl, self.table))
        T, n = int(qsl[-1]), int(lens.sum())
        slots, pos = self.slots.cpu().numpy(), self.pos.cpu().numpy()
        pool = f64(self.pool)
        # the append
        x, cs = f64(self.kv_new)[:T], self.cs.cpu().numpy()[pos[:T]]
        rows = pool.reshape(-1, 576)[slots[:T]]
        y = ref.norm(x[:, :512], f64(self.weight), 1e-6)
        close(rows[:, :512], y, ref.turned_bound(y, np.abs(y)))
        y, size = ref.rotate(x[:, None, 512:], cs, False)
        close(rows[:, 512:], y[:, 0], ref.turned_bound(y, size)[:, 0])
        y, size = ref.rotate(f64(before)[:T, :, 128:], cs, False)
        close(f64(self.q)[:T, :, 128:], y, ref.turned_bound(y, size))
        # the two forms, each over what it was given
        want, bound = ref.absorbed(f64(self.q_abs), pool, tab, lens, qsl, self.scale)
        lat = f64(self.lat)
        close(lat[:T], want[:T], bound[:T])
        kv, rope, kb = ref.expand(pool, f64(self.w), tab, lens)
        close(f64(self.kv)[:n], kv, kb)
        assert np.array_equal(f64(self.kr)[:n], rope)
        w2, b2 = ref.expanded(f64(self.q), f64(self.kv), f64(self.kr), lens, qsl, self.scale)
        out = f64(self.out)
        close(out[:T], w2[:T], b2[:T])
        assert (out[T:] == 7).all() and (lat[T:] == 7).all()
        self.agree(lat, out, bound, b2, kv, kb, lens, qsl, T)

    def agree(self, lat, out, b1, b2, kv, kb, lens, qsl, T):
        """W (absorbed) is the expanded form, within what each rounds on the way:
        the absorbed queries (half a step a number), the expanded keys and values (kb)."""
        w, q, qa, pool = f64(self.w), f64(self.q), f64(self.q_abs), f64(self.pool)
        got = np.einsum("thc,hdc->thd", lat, w[:, 128:])
        tol = np.einsum("thc,hdc->thd", b1, np.abs(w[:, 128:])) + b2
        k0 = 0
        for r, n in enumerate(lens):
            c = pool[self.table.cpu().numpy()[r, :ref.cdiv(n, 16)]].reshape(-1, 576)[:n, :512]
            for t in range(qsl[r], qsl[r + 1]):
                for h in range(self.H):
                    # a score off by d moves a mean of numbers |v| by (exp(2 d) - 1) mean |v|, at most their largest
                    d1 = self.scale * (2.0 ** -8 * np.abs(qa[t, h, :512]) * (1 + 2.0 ** -6) @ np.abs(c).T).max()
                    d2 = self.scale * (np.abs(q[t, h, :128]) @ kb[k0:k0 + n, h, :128].T).max()
                    v, vb = np.abs(kv[k0:k0 + n, h, 128:]).max(0), kb[k0:k0 + n, h, 128:].max(0)
                    tol[t, h] += (np.expm1(2 * d1) + np.expm1(2 * d2)) * v + vb
            k0 += n
        assert (np.abs(got - out)[:T] <= tol[:T]).all()
        # (and on the whole far nearer than that)
        assert np.abs(got - out)[:T].mean() < 0.02 * np.abs(out[:T]).mean()


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(graph):
    rng = np.random.default_rng(3)
    loop = Loop(R=6, cols=9, nb=40, cap=90, H=5, rows=6 * 144)
    lens, g = np.zeros(6, int), None
    for i in range(8):
        new = np.minimum(rng.choice([0, 1, 1, 2, 37], 6), 144 - lens)
        loop.inputs(new)
        before = loop.q.clone()
        if graph and g is None:
            loop.step()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                loop.step()
        elif graph:
            g.replay()
        else:
            loop.step()
        torch.cuda.synchronize()
        loop.check(before)
        lens = loop.lens.cpu().numpy()
        lens = np.where(rng.random(6) < 0.2, 0, np.maximum(lens - rng.integers(0, 4, 6), 0))
        loop.keep.copy_(torch.tensor(lens, dtype=I32))
        pkv.pkv_release_blocks(loop.table, loop.lens, loop.keep, loop.free, loop.nfree)
        loop.lens.copy_(loop.keep)


def test_norm_rope_append_then_attention():
    """The joint projection's rows through the call and into pkv_attention, step
    after step."""
    R, hq, hkv, cols = 5, 12, 2, 6
    g = torch.Generator().manual_seed(1)
    nb = R * cols
    i32 = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
    table, lens, free, nfree = i32(R, cols), i32(R), torch.arange(nb, dtype=I32, device="cuda"), i32(1) + nb
    pools = [torch.full((nb, hkv, 16, 128), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
    cs = torch.from_numpy(ref.table(96, 128)).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(128, generator=g)).to(BF).cuda() for _ in range(2))
    for new in ([20, 1, 0, 33, 7], [1, 1, 1, 1, 1], [1, 30, 5, 1, 0], [2, 2, 2, 2, 2]):
        T = sum(new)
        qsl, slots = i32(R + 1), torch.zeros(T, dtype=torch.int64, device="cuda")
        pkv.pkv_build_step(lens, dev(new, I32), free, nfree, table, lens, qsl, slots)
        qkv = torch.randn(T, hq + 2 * hkv, 128, generator=g).to(BF).cuda()
        pos = torch.cat([torch.arange(int(n) - m, int(n)) for n, m in zip(lens.cpu(), new)]).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        rot = pkv.pkv_norm_rope_append(q, k, v, pos, cs, slots, *pools, q_weight=wq, k_weight=wk)
        out = pkv.pkv_attention(rot, *pools, table, lens, qsl, 128 ** -0.5)
        y, size = ref.rotate(ref.norm(f64(q), f64(wq), 1e-6), cs.cpu().numpy()[pos.cpu().numpy()], False)
        close(rot, y, ref.turned_bound(y, size))
        tab, s = table.cpu().numpy(), 0
        for r, m in enumerate(new):
            n = int(lens[r])
            for h in range(hq if m else 0):
                kk, vv = (f64(p)[tab[r, :ref.cdiv(n, 16)], h * hkv // hq].reshape(-1, 128)[:n] for p in pools)
                sees = np.arange(n)[None, :] <= np.arange(n - m, n)[:, None]
                want, bound = ref._attend(f64(rot)[s:s + m, h], kk, vv, 128 ** -0.5, sees)
                close(f64(out)[s:s + m, h], want, bound)
            s += m


# ------------------------------------------------------------ graphs, streams
def _buffers(c):
    """The case's tensors on the device, to be called with again and again."""
    keys = ("tab", "lens", "qsl") if "tab" in c else ("lens", "qsl", "ksl")
    c["t"] = [dev(c[k], I32) for k in keys]
    c["out"] = torch.full((*c["q"].shape[:2], 512 if "tab" in c else 128), 7.0, dtype=BF, device="cuda")
    return c


def _call(c, **kw):
    if "tab" in c:
        return pkv.pkv_attention_latent(c["q"], c["pool"], *c["t"], c["scale"], out=c["out"], **kw)
    return pkv.pkv_attention_expanded(c["q"], c["kv"], c["kr"], *c["t"], c["scale"], out=c["out"], **kw)


def _capture(c, ws):
    _call(c, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(c, workspace=ws)
    return g


def test_graphs_that_share_a_workspace():
    """Different calls, captured with one workspace and replayed in turn."""
    ws = pkv.LatentWorkspace()
    cases = [_buffers(c) for c in (lat_case([3000, 20], [1, 1], 16), exp_case([2000], [50], 2), lat_case([50] * 200, [1] * 200, 8),
                                   exp_case([600] * 8, [512] * 8, 10), lat_case([700] * 4, [1] * 4, 128))]
    graphs = [_capture(c, ws) for c in cases]
    for c in cases:
        c["first"] = c["out"].clone()
        (lat_check if "tab" in c else exp_check)(c, c["first"])
    rng = np.random.default_rng(0)
    for i in rng.integers(0, len(cases), 60):
        cases[i]["out"].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(cases[i]["out"], cases[i]["first"])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_a_graph_serves_other_lengths(form):
    """Captured at one step, replayed at others: fewer requests in use, other lengths."""
    ws = pkv.LatentWorkspace()
    if form == "absorbed":
        make = lambda lens, qs, seed: lat_case(lens, qs, 16, seed=seed, pad=12 - sum(qs))  # noqa: E731
        steps = [([500, 40, 7], [4, 4, 4]), ([2000, 0, 1], [1, 0, 1]), ([3, 90, 600], [3, 1, 8]), ([0, 0, 0], [0, 0, 0])]
    else:
        make = lambda lens, qs, seed: exp_case(lens, qs, 3, seed=seed, pad=300 - sum(qs))  # noqa: E731
        steps = [([500, 400, 200], [100, 100, 100]), ([1000, 0, 100], [1, 0, 100]), ([3, 90, 1007], [3, 1, 256]),
                 ([1, 0, 0], [0, 0, 0])]
    c = make(*steps[0], 0)
    big = 140 if form == "absorbed" else 1100
    if form == "absorbed":
        c["pool"] = torch.full((big, 16, 576), float("nan"), dtype=BF, device="cuda")
        c["tab"] = np.full((3, big), 10 ** 8, np.int32)
    else:
        c["kv"] = torch.full((big, 3, 256), float("nan"), dtype=BF, device="cuda")
        c["kr"] = torch.full((big, 64), float("nan"), dtype=BF, device="cuda")
    _buffers(c)
    for t in c["t"]:
        t.zero_()  # (nothing to do: only the capture's shapes count)
    g = _capture(c, ws)
    for i, (lens, qs) in enumerate(steps):
        n = make(lens, qs, 5 + i)
        c["out"].fill_(7.0)
        c["q"].copy_(n["q"])
        if form == "absorbed":
            k = n["pool"].shape[0]
            c["pool"].fill_(float("nan"))
            c["pool"][:k] = n["pool"]
            c["t"][0].fill_(10 ** 8)
            c["t"][0][:, :n["tab"].shape[1]] = dev(n["tab"], I32)
        else:
            k = n["kv"].shape[0]
            c["kv"][:k], c["kr"][:k] = n["kv"], n["kr"]
            c["t"][2].copy_(dev(n["ksl"], I32))
        c["t"][1 if form == "absorbed" else 0].copy_(dev(lens, I32))
        c["t"][2 if form == "absorbed" else 1].copy_(dev(n["qsl"], I32))
        g.replay()
        (lat_check if form == "absorbed" else exp_check)(n, c["out"])
        assert (c["out"][sum(qs):] == 7).all()


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own."""
    cases = [_buffers(c) for c in (lat_case([4000, 900], [1, 1], 16), lat_case([5000], [3], 64), exp_case([1500], [200], 2),
                                   exp_case([600] * 8, [512] * 8, 10))]
    spaces, streams = [pkv.LatentWorkspace() for _ in cases], [torch.cuda.Stream() for _ in cases]
    for c in cases:
        _call(c)
        c["first"] = c["out"].clone()
        (lat_check if "tab" in c else exp_check)(c, c["first"])
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, s in zip(cases, spaces, streams):
            _call(c, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c["out"], c["first"])


def test_requests_may_share_blocks():
    c = lat_case([64, 70], [1, 2], 20)
    c["tab"][1, :4] = c["tab"][0, :4]
    lat_check(c, lat_run(c))
    w = (torch.randn(2, 256, 512) / 20).to(BF).cuda()
    kv, kr = torch.empty(134, 2, 256, dtype=BF, device="cuda"), torch.empty(134, 64, dtype=BF, device="cuda")
    pkv.pkv_expand_latent(c["pool"], w, dev(c["tab"], I32), dev(c["lens"], I32), dev([0, 64, 134], I32), kv, kr)
    want, rope, bound = ref.expand(f64(c["pool"]), f64(w), c["tab"], c["lens"])
    close(kv, want, bound)
    assert torch.equal(kv[:64], kv[64:128]) and np.array_equal(f64(kr), rope)


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_queries_that_are_not_finite_spoil_their_rows_only(what):
    for c, run, check in ((lat_case([200, 3000], [3, 1], 16), lat_run, lat_check), (lat_case([900] * 3, [1] * 3, 128), lat_run, lat_check),
                          (exp_case([130, 300], [130, 70], 3), exp_run, exp_check), (exp_case([2000], [50], 2), exp_run, exp_check),
                          (exp_case([600] * 8, [512] * 8, 10), exp_run, exp_check)):
        good = run(c).clone()
        T, H = c["q"].shape[:2]
        for t, h in ((0, 0), (T // 2, H // 2), (T - 1, H - 1)):
            c["q"][t, h, 3] = float(what)
        out = run(c)
        rows = torch.ones(T, H, dtype=torch.bool, device="cuda")
        for t, h in ((0, 0), (T // 2, H // 2), (T - 1, H - 1)):
            rows[t, h] = False
        assert torch.equal(out[rows], good[rows])
        check(c, out)


def test_requests_of_a_step_mostly_idle():
    """Far more requests than rows, most without query tokens, some without keys."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 200, 700).tolist()
    qs = [0] * 700
    for r, m in ((3, 1), (350, 5), (699, 2)):
        lens[r], qs[r] = 150 + r, m
    c = lat_case(lens, qs, 16)
    lat_check(c, lat_run(c))
    e = exp_case(lens, qs, 2)
    exp_check(e, exp_run(e))


def test_pairs_ignore_what_others_hold():
    """Whole pairs of query tiles over keys between rows of NaN, requests of odd lengths."""
    lens, qs = [333, 700, 129, 512], [333, 600, 129, 512]
    c = exp_case(lens, qs, 26)
    assert sum(qs) >= 192 * 4
    assert sum(qs) * 26 >= 256 * torch.cuda.get_device_properties(0).multi_processor_count
    want = exp_run(c).clone()
    exp_check(c, want)
    a, b = 333, 333 + 700  # the second request's rows
    c["kv"][a:b], c["kr"][a:b] = float("nan"), float("nan")
    pad = torch.full((300, 26, 256), float("nan"), dtype=BF, device="cuda")
    c["kv"], c["kr"] = torch.cat([c["kv"], pad]), torch.cat([c["kr"], pad[:, 0, :64].contiguous()])
    out = exp_run(c)
    assert torch.equal(out[:333], want[:333]) and torch.equal(out[933:], want[933:])
    assert torch.isnan(out[333:933]).all()


def test_workspaces_that_are_too_small_are_refused():
    c, e = _buffers(lat_case([40], [1], 16)), _buffers(exp_case([40], [3], 2))
    ws = pkv.LatentWorkspace()
    ws.nbytes -= 1
    for x in (c, e):
        with pytest.raises(pkv.PagedKVError) as err:
            _call(x, workspace=ws)
        assert err.value.code == pkv._binding.PKV_ERR_WORKSPACE
        assert (x["out"] == 7).all()


def test_capture_without_a_workspace():
    """The call's own workspace is captured with it."""
    for c, check in ((_buffers(lat_case([3000, 20], [1, 1], 16)), lat_check), (_buffers(exp_case([2000], [50], 2)), exp_check)):
        _call(c)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(c)
            _call(c)
        for _ in range(3):
            c["out"].fill_(7.0)
            g.replay()
            check(c, c["out"])


def _offset(t):
    """The same tensor 16 bytes behind a 32-byte boundary."""
    b = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)[8:].view(t.shape)
    return b.copy_(t)


def test_buffers_need_16_bytes_of_alignment_only():
    for c in (exp_case([130, 40], [130, 7], 3), exp_case([2000], [50], 2), exp_case([600] * 8, [512] * 8, 10)):
        want = exp_run(c)
        for k in ("q", "kv", "kr"):
            c[k] = _offset(c[k])
        out = _offset(torch.zeros_like(want))
        assert out.data_ptr() % 32 == 16
        assert torch.equal(exp_run(c, out=out), want)
    for c in (lat_case([3000, 20], [1, 3], 16), lat_case([700] * 4, [1] * 4, 128)):
        want = lat_run(c)
        c["q"], c["pool"] = _offset(c["q"]), _offset(torch.nan_to_num(c["pool"]))
        assert torch.equal(lat_run(c, out=_offset(torch.zeros_like(want))), want)
    c, w = lat_case([300], [1], 1), (torch.randn(3, 256, 512, device="cuda") / 20).to(BF)
    outs = []
    for f in (lambda t: t, _offset):
        kv, kr = f(torch.zeros(300, 3, 256, dtype=BF, device="cuda")), f(torch.zeros(300, 64, dtype=BF, device="cuda"))
        pkv.pkv_expand_latent(f(c["pool"]), f(w), dev(c["tab"], I32), dev(c["lens"], I32), dev([0, 300], I32), kv, kr)
        outs.append((kv, kr))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_empty_calls():
    none = torch.empty(0, 16, 576, dtype=BF, device="cuda")
    pool = torch.zeros(3, 16, 576, dtype=BF, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
    assert pkv.pkv_attention_latent(none, pool, i32(2, 3), i32(2), i32(3), 0.1).shape == (0, 16, 512)
    assert pkv.pkv_attention_latent(none, pool, i32(0, 3), i32(0), i32(1), 0.1).shape == (0, 16, 512)
    q, kv, kr = none[..., :192].contiguous(), torch.empty(0, 16, 256, dtype=BF, device="cuda"), torch.empty(0, 64, dtype=BF, device="cuda")
    assert pkv.pkv_attention_expanded(q, kv, kr, i32(2), i32(3), i32(3), 0.1).shape == (0, 16, 128)
    pkv.pkv_expand_latent(pool, torch.empty(16, 256, 512, dtype=BF, device="cuda"), i32(2, 3), i32(2), i32(3), kv, kr)
    long = torch.zeros(0, dtype=torch.int64, device="cuda")
    pkv.pkv_append_latent(none[:, 0], long, torch.zeros(4, 64, device="cuda"), long, pool)
    assert (pool == 0).all()


# ------------------------------------------------------------ far ends
def test_blocks_past_2_32_elements():
    nb = (1 << 32) // (16 * 576) + 40
    pool = torch.empty(nb, 16, 576, dtype=BF, device="cuda")
    c = lat_case([100, 35], [1, 2], 16)
    k = c["pool"].shape[0]
    pool[-k:] = c["pool"]
    c["tab"] = np.where(c["tab"] < k, c["tab"] + nb - k, c["tab"])
    small, c["pool"] = c["pool"], pool
    got = lat_run(c)
    low = dict(c, pool=small, tab=np.where(c["tab"] < nb, c["tab"] - (nb - k), c["tab"]))
    lat_check(low, got)
    w = (torch.randn(2, 256, 512) / 20).to(BF).cuda()
    outs = []
    for p, t in ((pool, c["tab"]), (small, low["tab"])):
        kv, kr = torch.empty(135, 2, 256, dtype=BF, device="cuda"), torch.empty(135, 64, dtype=BF, device="cuda")
        pkv.pkv_expand_latent(p, w, dev(t, I32), dev(c["lens"], I32), dev([0, 100, 135], I32), kv, kr)
        outs.append((kv, kr))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    kv = torch.randn(3, 576, device="cuda").to(BF)
    slots = torch.tensor([nb * 16 - 1, nb * 16 - 17, nb * 16 - 40], device="cuda")
    pos, cs = torch.arange(3, device="cuda"), torch.from_numpy(ref.table(8, 64)).cuda()
    pkv.pkv_append_latent(kv, pos, cs, slots, pool)
    assert torch.equal(pool.view(-1, 576)[slots][:, :512], kv[:, :512])
    y, size = ref.rotate(f64(kv)[:, None, 512:], cs.cpu().numpy()[:3], False)
    close(pool.view(-1, 576)[slots][:, 512:], y[:, 0], ref.turned_bound(y, size)[:, 0])


def test_keys_past_2_32_elements_of_kv():
    H, far = 128, (1 << 32) // (128 * 256) + 100
    c = exp_case([40, 70], [1, 30], H)
    n = far + 110
    kv, kr = torch.empty(n, H, 256, dtype=BF, device="cuda"), torch.empty(n, 64, dtype=BF, device="cuda")
    kv[far:], kr[far:] = c["kv"], c["kr"]
    lens, ksl = [far, 40, 70], [0, far, far + 40, n]
    out = pkv.pkv_attention_expanded(c["q"], kv, kr, dev(lens, I32), dev([0, 0, 1, 31], I32), dev(ksl, I32), c["scale"])
    exp_check(c, out)
    # and expanded there: a request that fills the rows before, two behind it
    small = lat_case([far, 40, 70], [1, 1, 1], 1)
    w = (torch.randn(H, 256, 512) / 20).to(BF).cuda()
    kv.fill_(7.0)
    pkv.pkv_expand_latent(small["pool"], w, dev(small["tab"], I32), dev(lens, I32), dev(ksl, I32), kv, kr)
    rows = [0, 1, far - 1, far, far + 39, far + 40, n - 1]
    at = [(0, 0), (0, 1), (0, far - 1), (1, 0), (1, 39), (2, 0), (2, 69)]
    c0 = torch.stack([small["pool"][small["tab"][r, j // 16], j % 16] for r, j in at])
    want = np.einsum("jc,hoc->jho", f64(c0)[:, :512], f64(w), optimize=True)
    size = np.einsum("jc,hoc->jho", np.abs(f64(c0)[:, :512]), np.abs(f64(w)), optimize=True)
    close(kv[rows], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size)
    assert torch.equal(kr[rows], c0[:, 512:])


def test_norm_rope_pools_past_2_32_elements():
    hkv = 8
    nb = (1 << 32) // (hkv * 16 * 128) + 20
    pools = [torch.empty(nb, hkv, 16, 128, dtype=BF, device="cuda") for _ in range(2)]
    qkv = torch.randn(4, 2 + 2 * hkv, 128, device="cuda").to(BF)
    slots = torch.tensor([nb * 16 - 1, nb * 16 - 30, 5, nb * 16 - 100], device="cuda")
    pos, cs = torch.arange(4, device="cuda"), torch.from_numpy(ref.table(8, 128)).cuda()
    k, v = qkv[:, 2:2 + hkv], qkv[:, 2 + hkv:]
    pkv.pkv_norm_rope_append(qkv[:, :2], k, v, pos, cs, slots, *pools)
    y, size = ref.rotate(f64(k), cs.cpu().numpy()[:4], False)
    close(pools[0][slots // 16, :, slots % 16], y, ref.turned_bound(y, size))
    assert torch.equal(pools[1][slots // 16, :, slots % 16], v)


# ------------------------------------------------------------ refusals of the binding
def test_the_binding_refuses():
    c, e = lat_case([40, 5], [1, 1], 16), exp_case([40, 5], [1, 5], 2)
    t, u = [dev(c[k], I32) for k in ("tab", "lens", "qsl")], [dev(e[k], I32) for k in ("lens", "qsl", "ksl")]
    q, pool = c["q"], c["pool"]
    wide = torch.zeros(2, 16, 1152, dtype=BF, device="cuda")

    def no(call, *a, error=(ValueError, TypeError, pkv.PagedKVError), **kw):
        with pytest.raises(error):
            call(*a, **kw)

    lat, s = pkv.pkv_attention_latent, 0.1
    no(lat, q.half(), pool, *t, s)
    no(lat, wide[..., :576], pool, *t, s)  # rows apart
    no(lat, q, pool.float(), *t, s)
    no(lat, q, pool, t[0].long(), *t[1:], s)
    no(lat, q, pool, t[0], t[1][:1], t[2], s)
    no(lat, q, pool, *t[:2], t[2][:2], s)
    no(lat, q, pool[..., :512].contiguous(), *t, s)
    no(lat, q, pool, *t, s, out=torch.empty(2, 16, 576, dtype=BF, device="cuda"))
    no(lat, q, pool, *t, s, workspace=object())
    no(lat, torch.zeros(2, 129, 576, dtype=BF, device="cuda"), pool, *t, s)
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        no(lat, q, pool, *t, bad)
        no(pkv.pkv_attention_expanded, e["q"], e["kv"], e["kr"], *u, bad)
    exp = pkv.pkv_attention_expanded
    no(exp, e["q"][..., :128].contiguous(), e["kv"], e["kr"], *u, s)
    no(exp, e["q"], e["kv"][:, :1].contiguous(), e["kr"], *u, s)
    no(exp, e["q"], e["kv"], e["kr"][:-1], *u, s)
    no(exp, e["q"], e["kv"], e["kr"], u[0], u[1], u[2][:2], s)
    no(exp, e["q"], e["kv"], e["kr"], *u, s, out=torch.empty_like(e["q"]))
    w, kv, kr = torch.zeros(2, 256, 512, dtype=BF, device="cuda"), e["kv"], e["kr"]
    no(pkv.pkv_expand_latent, pool, w[:, :255].contiguous(), t[0], t[1], t[2], kv, kr)
    no(pkv.pkv_expand_latent, pool, w[:1], t[0], t[1], t[2], kv, kr)
    no(pkv.pkv_expand_latent, pool, w, t[0], t[1], t[1], kv, kr)
    i64, cs = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(4, 64, device="cuda")
    rows, qr = torch.zeros(2, 576, dtype=BF, device="cuda"), torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    app = pkv.pkv_append_latent
    no(app, rows[:, :512], i64, cs, i64, pool)
    no(app, rows, i64[:1], cs, i64, pool)
    no(app, rows, i64, cs[:, :32].contiguous(), i64, pool)
    no(app, rows, i64, cs, i64, pool, weight=rows[0])
    no(app, rows, i64, cs, i64, pool, q_rope=qr[:1])
    no(app, rows, i64, cs, i64, pool, q_rope_out=qr)
    no(app, rows, i64, cs, i64, pool, q_rope=qr, q_rope_out=qr.float())
    flat = torch.zeros(1024, dtype=BF, device="cuda")
    no(app, rows, i64, cs, i64, pool, q_rope=qr, q_rope_out=flat[:64].expand(2, 4, 64))
    no(app, rows, i64, cs, i64, pool, q_rope=flat[:512].view(2, 4, 64), q_rope_out=flat[64:576].view(2, 4, 64))
    no(app, rows, i64, cs, i64, pool, weight=torch.ones(512, dtype=BF, device="cuda"), eps=0.0)
    pools = [torch.zeros(2, 1, 16, 128, dtype=BF, device="cuda") for _ in range(2)]
    x, one = torch.zeros(2, 4, 128, dtype=BF, device="cuda"), torch.zeros(2, 1, 128, dtype=BF, device="cuda")
    nra, cs = pkv.pkv_norm_rope_append, torch.zeros(4, 128, device="cuda")
    no(nra, x, one, one[:1], i64, cs, i64, *pools)
    no(nra, x, x, x, i64, cs, i64, *pools)
    no(nra, x[..., :64], one, one, i64, cs, i64, *pools)
    no(nra, x, one, one, i64, cs[:, :24].contiguous(), i64, *pools)
    no(nra, x, one, one, i64, cs, i64, pools[0], pools[1][:1])
    no(nra, x, one, one, i64, cs, i64, *pools, q_weight=torch.ones(64, dtype=BF, device="cuda"))
    big = torch.zeros(2, 6, 128, dtype=BF, device="cuda")
    no(nra, big[:, :4], big[:, 4:5], big[:, 5:], i64, cs, i64, *pools, q_out=big[:, 1:5])
    assert (pool[c["tab"][0, 0], 0].float() - lat_case([40, 5], [1, 1], 16)["pool"][c["tab"][0, 0], 0].float()).abs().max() == 0
