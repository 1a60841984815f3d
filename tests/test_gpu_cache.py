"""The paged 4-bit history cache on the GPU against plain 64-bit forms
(tests/cache_ref.py): stored bytes and read rows bit for bit, plans as whole
numbers, attention within the bound derived in cache_ref.attend."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from sparse_hstu_attention_b200 import SLAError, _abi, cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def offs_of(rows):
    return dev32(np.concatenate([[0], np.cumsum(rows)]))


def silu_rows(T, H, d, seed, strided=True):
    """q, k, v [T, H, d] bf16 on the CPU, as column blocks of one projection."""
    g = torch.Generator().manual_seed(seed)
    x = torch.nn.functional.silu(torch.randn((max(T, 1), 4 * H * d), generator=g)).bfloat16()[:T]
    q, k, v = (x[:, i * H * d:(i + 1) * H * d].reshape(T, H, d) for i in (2, 3, 1))
    return q, k, v


def on_gpu(x, wide):
    """x on the GPU; `wide`: as a view into rows 4 times as long."""
    T, H, d = x.shape
    if not wide:
        return x.to(DEV)
    buf = torch.full((T, 4 * H * d), float("nan"), dtype=x.dtype, device=DEV)
    out = buf[:, H * d:2 * H * d].unflatten(1, (H, d))
    out.copy_(x)
    return out


def tables_of(lengths, ps, seed, spare=3, most=None):
    """Tables whose sequence b holds lengths[b] tokens in pages drawn at random;
    the host copy beside the GPU's."""
    g = np.random.default_rng(seed)
    used = [-(-n // ps) for n in lengths]
    M = max(1, most or max(used))
    P = max(1, sum(used) + spare)
    perm = g.permutation(P)
    bt = g.integers(0, 2 ** 31 - 1, size=(len(lengths), M))  # unused entries are garbage
    at = P - sum(used)
    free = perm[:at]
    for b, n in enumerate(used):
        bt[b, :n] = perm[at:at + n]
        at += n
    t = cache.allocate_tables(len(lengths), M, P, page_size=ps, device=DEV)
    t.lengths.copy_(dev32(lengths))
    t.block_table.copy_(torch.from_numpy(bt.astype(np.int32)))
    t.free_pages[:len(free)] = torch.from_numpy(free.astype(np.int32)).to(DEV)
    t.free_count.fill_(len(free))
    return t, ref.Tables(lengths, bt, free, P, ps)


# ------------------------------------------------------------ append and read
@pytest.mark.parametrize("H,d,ps,T", [(1, 32, 16, 1), (2, 64, 32, 7), (3, 128, 64, 130),
                                      (4, 128, 16, 333), (2, 32, 64, 4100), (1, 64, 16, 17),
                                      (40, 128, 64, 700)])
@pytest.mark.parametrize("order", ["runs", "mixed"])
def test_append_and_read(H, d, ps, T, order):
    """Every byte of the pages as the plain form has it, the untouched ones as
    they were; rows read back are m + s code in bf16."""
    g = np.random.default_rng(T)
    P = T // ps + 4
    if order == "runs":  # sequences of consecutive slots, starting anywhere
        slots, s = [], int(g.integers(0, ps))
        while len(slots) < T and s < P * ps:
            n = int(g.integers(1, 200))
            slots += list(range(s, min(s + n, P * ps)))
            s += n + int(g.integers(0, 3))
        slots = slots[:T] + [-1] * max(0, T - len(slots))
    else:
        slots = g.permutation(P * ps)[:T].tolist()
    slots = torch.tensor(slots)
    if T > 5:
        slots[g.integers(0, T, 3)] = -1
    _, k, v = silu_rows(T, H, d, T)
    k[0] = 0.5           # no range: step 0
    if T > 5:
        k[3, 0, 1], v[4, 0, 2], v[5, 0, 0] = float("nan"), float("inf"), -float("inf")
        v[1], k[2] = v[1] * 1e-39, k[2] * 1e30   # steps that vanish, and large ones
        k[1, 0, 0], k[1, 0, 1] = 3e38, -3e38     # a range beyond fp32
    pages = torch.from_numpy(g.integers(0, 256, size=(P, H, ps * (d + 8)), dtype=np.uint8))
    want = ref.pack(pages.clone(), ps, slots, k, v)
    t = cache.allocate_tables(1, 1, P, page_size=ps, device=DEV)
    got = pages.to(DEV)
    cache.append(on_gpu(k, True), on_gpu(v, T % 2 == 0), slots.to(DEV), got, t)
    kept = [s for s in slots.tolist() if s >= 0]
    # a NaN pair may have any NaN's bits: compare it as NaN, everything else as bytes
    K0, V0 = ref.unpack(want, ps, d)
    K1, V1 = ref.unpack(got, ps, d)
    for x, y in ((K0, K1), (V0, V1)):
        x, y = x.reshape(-1, H, d)[kept], y.reshape(-1, H, d)[kept]
        assert torch.equal(x.isnan(), y.isnan())
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    odd = (got.cpu() != want).sum().item()
    assert odd <= 6 * 4  # at most the bytes of the few NaN pairs
    rk, rv = cache.read(slots.to(DEV), got, t)
    for x, y in ((K0, rk), (V0, rv)):
        x = x.reshape(-1, H, d)[slots.clamp(min=0)]
        x[slots < 0] = 0
        y = y.cpu().double()
        assert torch.equal(x.isnan(), y.isnan())
        assert torch.equal(x.float().bfloat16().double().nan_to_num(), y.nan_to_num())
    assert cache.get_error(t) == 0


def test_slots_beyond_the_pages_are_reported_and_write_nothing():
    t = cache.allocate_tables(1, 1, 3, page_size=16, device=DEV)
    pages = torch.full((3, 1, 16 * 40), 77, dtype=torch.uint8, device=DEV)
    _, k, v = (x.to(DEV) for x in silu_rows(2, 1, 32, 0))
    cache.append(k, v, torch.tensor([48, 1 << 40], device=DEV), pages, t)
    assert cache.get_error(t) == _abi.ERR_BAD_INPUT
    assert bool((pages == 77).all())
    cache.append(k, v, torch.tensor([0, 1], device=DEV), pages, t)  # still set: nothing is done
    assert bool((pages == 77).all())


# ---------------------------------------------------------------------- plan
def check_plan(t, host, rows, cand, release, pad=0):
    T = int(sum(rows))
    slots = cache.plan(t, offs_of(rows), dev32(cand) if any(cand) else None, total_tokens=T + pad,
                       release=dev32(release) if any(release) else None)
    want = host.plan(rows, cand, release, T + pad)
    assert cache.get_error(t) == 0
    assert slots.tolist() == want
    assert t.lengths.tolist() == host.lengths
    assert int(t.free_count) == host.count
    assert t.free_pages.tolist()[:host.count] == host.stack[:host.count]
    assert t.block_table.tolist() == host.bt
    return slots


@pytest.mark.parametrize("B,ps,most,seed", [(1, 64, 1, 0), (5, 16, 40, 1), (64, 32, 3, 2),
                                            (1500, 16, 20, 3), (3, 64, 9000, 4),
                                            (2500, 32, 60, 5)])
def test_plan_matches_a_walk(B, ps, most, seed):
    """Several steps in a row: appends, candidates, rows behind the last
    sequence, slots that change hands (one block up to 8192 rows, a grid above)."""
    g = np.random.default_rng(seed)
    lengths = g.integers(0, 3 * ps, size=B).tolist()
    M = -(-(3 * ps + 3 * most) // ps) + 1
    t, host = tables_of(lengths, ps, seed, spare=B * (2 + 3 * most // ps), most=M)
    for step in range(3):
        fresh = np.where(g.random(B) < 0.7, g.integers(0, most, size=B, endpoint=True), 0)
        cand = np.where(g.random(B) < 0.5, g.integers(0, 5, size=B), 0) * (step > 0)
        release = (g.random(B) < 0.3) * (step == 2)
        check_plan(t, host, (fresh + cand).tolist(), cand.tolist(), release.astype(int).tolist(),
                   pad=7 * step)


def test_plan_without_pages_changes_nothing():
    for total in (0, 20000):  # one block, and the grid
        t, _ = tables_of([10, 20, 30], 16, 1, spare=2, most=4000)
        before = t.buf.clone()
        rows = [20, 20, 20 + total]
        slots = cache.plan(t, offs_of(rows), total_tokens=sum(rows))
        assert cache.get_error(t) == _abi.ERR_NO_PAGES
        assert bool((slots == -1).all())
        assert torch.equal(t.buf[16:], before[16:])
        # the other calls do nothing until a plan succeeds
        pages = torch.full((t.num_pages, 1, 16 * 40), 5, dtype=torch.uint8, device=DEV)
        out = torch.full((60 + total, 1, 32), 7.0, dtype=torch.bfloat16, device=DEV)
        q, k, v = (x.to(DEV) for x in silu_rows(60 + total, 1, 32, 0))
        cache.append(k, v, torch.arange(60 + total, device=DEV) % 40, pages, t)
        assert bool((pages == 5).all())
        slots = cache.plan(t, offs_of([1, 0, 0]), total_tokens=1)
        assert cache.get_error(t) == 0 and int(slots[0]) >= 0


@pytest.mark.parametrize("what", ["down", "past", "first", "targets", "long", "length", "count"])
def test_plan_refuses_bad_inputs(what):
    t, _ = tables_of([10, 20], 16, 1, spare=9, most=4)
    offs, nt = [0, 3, 6], [0, 1]
    if what == "down":
        offs = [0, 5, 3]
    if what == "past":
        offs = [0, 3, 9]
    if what == "first":
        offs = [1, 3, 6]
    if what == "targets":
        nt = [0, 4]
    if what == "long":
        offs = [0, 55, 55]
    if what == "length":
        t.lengths[1] = -4
    if what == "count":
        t.free_count.fill_(t.num_pages + 1)
    before = t.buf.clone()
    T = 55 if what == "long" else 6
    nt = [0, 0] if what == "long" else nt
    slots = cache.plan(t, dev32(offs), dev32(nt), total_tokens=T)
    assert cache.get_error(t) == _abi.ERR_BAD_INPUT
    assert bool((slots == -1).all()) and torch.equal(t.buf[16:], before[16:])


def test_slot_map_gives_the_last_tokens():
    lengths = [40, 0, 7, 130]
    t, host = tables_of(lengths, 32, 3)
    rows = [33, 0, 7, 64]
    slots = cache.slot_map(t, offs_of(rows), total_tokens=sum(rows) + 3).tolist()
    want = []
    for b, n in enumerate(rows):
        want += [host.bt[b][p // 32] * 32 + p % 32 for p in range(lengths[b] - n, lengths[b])]
    assert slots == want + [-1] * 3 and cache.get_error(t) == 0
    slots = cache.slot_map(t, offs_of([41, 0, 0, 1]), total_tokens=42).tolist()
    assert slots[:41] == [-1] * 41 and cache.get_error(t) == _abi.ERR_BAD_INPUT


# -------------------------------------------------------------------- attend
def filled(lengths, H, d, ps, seed, garbage=True):
    """Tables and pages holding random histories; per sequence the codes and
    pairs, token by token.  Unused bytes are garbage (NaN pairs among them)."""
    t, host = tables_of(lengths, ps, seed)
    g = torch.Generator().manual_seed(seed)
    pages = torch.full((t.num_pages, H, ps * (d + 8)), 255 if garbage else 0, dtype=torch.uint8)
    tokens = []
    for b, n in enumerate(lengths):
        _, k, v = silu_rows(n, H, d, seed * 100 + b)
        slots = torch.tensor([host.bt[b][p // ps] * ps + p % ps for p in range(n)],
                             dtype=torch.int64)
        if n:
            pages = ref.pack(pages, ps, slots, k, v)
        tokens.append(tuple((c.double(), s, m) for c, s, m in (ref.quantise(k), ref.quantise(v)))
                      if n else ((torch.zeros(0, H, d).double(), torch.zeros(0, H).double(),
                                  torch.zeros(0, H).double()),) * 2)
    return t, pages.to(DEV), tokens


def run_attend(t, pages, tokens, lengths, rows, cand, H, d, seed, *, K1, K2, ctx, max_new=None,
               pad=0, wide=True, edit=None):
    T = int(sum(rows))
    q, k, v = silu_rows(T, H, d, seed + 1)
    if edit:
        edit(q, k, v)
    alpha, N = d ** -0.5, 100.0
    out = torch.full((T + pad, H, d), 3.0, dtype=torch.bfloat16, device=DEV)
    more = torch.full((pad, H, d), float("nan")).bfloat16()
    qg, kg, vg = (on_gpu(torch.cat([x, more]), wide) for x in (q, k, v))
    has = any(cand)
    cache.attend(qg, kg if has else None, vg if has else None, offs_of(rows),
                 dev32(cand) if has else None, pages, t, contextual_len=ctx, K1=K1, K2=K2,
                 alpha=alpha, N=N, max_new=max_new, out=out)
    assert cache.get_error(t) == 0
    assert bool((out[T:] == 3.0).all())
    want, tol = ref.attend(q, k, v, rows, cand, lengths, tokens, K1=K1, K2e=max(K2, ctx),
                           alpha=alpha, N=N)
    return out[:T].cpu().double(), want, tol


def check(got, want, tol):
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))


FEW = [([300], [1], [0]), ([0, 5, 64, 65, 700], [3, 1, 1, 2, 0], [3, 0, 1, 0, 0]),
       ([128, 1, 17], [16, 1, 33], [4, 0, 33]), ([2100, 900], [1, 1], [0, 0])]
MANY = [([200], [65], [0]), ([500, 3, 0], [130, 40, 33], [2, 40, 33]),
        ([300, 129, 128], [300, 129, 1], [0, 0, 0]), ([1000, 260], [150, 300], [150, 270])]


HEADS = [(2, 32, 16), (1, 64, 32), (3, 128, 64), (1, 128, 16), (2, 64, 64), (2, 32, 32)]
WINDOWS = [(1 << 20, 0, 0), (100, 20, 33), (0, 0, 0), (1, 0, 0), (0, 70, 0)]


@pytest.mark.parametrize("case,heads,window",
                         [(c, h, w) for c in range(8) for h in HEADS for w in WINDOWS
                          if c < 4 or h not in HEADS[4:] or w == WINDOWS[1]])
def test_attend(case, heads, window):
    (H, d, ps), (K1, K2, ctx) = heads, window
    lengths, rows, cand = (FEW + MANY)[case]
    t, pages, tokens = filled(lengths, H, d, ps, case + 1)
    got, want, tol = run_attend(t, pages, tokens, lengths, rows, cand, H, d, case, K1=K1, K2=K2,
                                ctx=ctx, max_new=max(rows), pad=case % 3, wide=case % 2 == 0)
    check(got, want, tol)
    if K1 == K2 == ctx == 0:  # history rows see nothing
        at = 0
        for n, c in zip(rows, cand):
            assert bool((got[at:at + n - c] == 0).all())
            at += n


def test_what_is_masked_does_not_reach_a_row():
    """NaN and infinities in tokens outside the window, in other candidates'
    rows and behind the length change nothing."""
    H, d, ps = 2, 64, 32
    lengths, K1 = [200, 300], 50
    for rows, cand in (([3, 4], [2, 4]), ([80, 70], [60, 65])):
        t, pages, tokens = filled(lengths, H, d, ps, 9)
        q, k, v = silu_rows(sum(rows), H, d, 10)
        args = dict(contextual_len=0, K1=K1, K2=0, alpha=0.1, N=10.0, max_new=max(rows))
        offs, nts = offs_of(rows), dev32(cand)
        qg, kg, vg = q.to(DEV), k.to(DEV), v.to(DEV)
        clean = cache.attend(qg, kg, vg, offs, nts, pages, t, **args)
        # tokens below every row's window become NaN, one candidate's row too
        slots = []
        for b, L in enumerate(lengths):
            low = L - (rows[b] - cand[b]) - K1
            slots += [int(t.block_table[b, p // ps]) * ps + p % ps for p in range(max(0, low))]
        bad = torch.full((len(slots), H, d), float("nan")).bfloat16().to(DEV)
        cache.append(bad, bad, torch.tensor(slots, device=DEV), pages, t)
        last = sum(rows) - 1
        kg[last], vg[last] = float("nan"), float("inf")
        got = cache.attend(qg, kg, vg, offs, nts, pages, t, **args)
        assert torch.equal(got[:last], clean[:last])
        assert bool(got[last].isnan().all())


@pytest.mark.parametrize("rows", [1, 70])
def test_pages_far_apart(rows):
    """Page offsets beyond 32 bits."""
    H, d, ps = 1, 128, 64
    lengths = [150, 90]
    t, pages, tokens = filled(lengths, H, d, ps, 4)
    stride = (1 << 30) + 256
    buf = torch.empty(stride * (t.num_pages - 1) + pages[0].numel(), dtype=torch.uint8,
                      device=DEV)
    far = torch.as_strided(buf, pages.shape, (stride, ps * (d + 8), 1))
    far.copy_(pages)
    got, want, tol = run_attend(t, far, tokens, lengths, [rows, rows], [0, 0], H, d, 1, K1=1 << 20,
                                K2=0, ctx=0, max_new=rows)
    check(got, want, tol)
    slots = cache.slot_map(t, offs_of([5, 5]), total_tokens=10)
    for x, y in zip(cache.read(slots, far, t), cache.read(slots, pages, t)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("what", ["page", "length", "offsets", "targets", "rows"])
@pytest.mark.parametrize("n", [1, 70])
def test_attend_reports_bad_inputs(what, n):
    H, d, ps = 2, 32, 16
    t, pages, _ = filled([160, 180], H, d, ps, 5, garbage=False)
    q, k, v = (x.to(DEV) for x in silu_rows(2 * n, H, d, 0))
    offs, nts, most = [0, n, 2 * n], [0, 1], n
    if what == "page":
        t.block_table[1, 2] = t.num_pages
    if what == "length":
        t.lengths[0] = 1 << 20
    if what == "offsets":
        offs = [0, n, 2 * n + 1]
    if what == "targets":
        nts = [0, n + 1]
    if what == "rows":
        offs, most = [0, 0, 2 * n], n
    out = cache.attend(q, k, v, dev32(offs), dev32(nts), pages, t, contextual_len=0, K1=1 << 20,
                       K2=0, alpha=0.1, N=10.0, max_new=most)
    assert out.shape == q.shape and cache.get_error(t) == _abi.ERR_BAD_INPUT


# ------------------------------------------------------------------ together
def test_a_serving_run():
    """Steps as a server makes them: histories come in whole, users bring single
    events and candidates, one slot changes hands; every output against the
    plain form over what was stored."""
    H, d, ps, B, K1, K2, ctx = 2, 64, 32, 4, 60, 20, 4
    t = cache.allocate_tables(B, 12, 40, page_size=ps, device=DEV)
    pages = [cache.allocate_pages(40, H, d, ps, DEV) for _ in range(2)]
    kept = [[None] * B for _ in pages]
    lengths = [0] * B
    steps = [([150, 70, 0, 33], [0, 0, 0, 0], [0] * 4), ([1, 1, 0, 1], [0, 0, 0, 0], [0] * 4),
             ([20, 9, 6, 0], [20, 8, 6, 0], [0] * 4), ([90, 0, 40, 2], [0, 0, 10, 1], [1, 0, 0, 0]),
             ([1, 2, 1, 18], [0, 1, 0, 18], [0] * 4)]
    for n, (rows, cand, release) in enumerate(steps):
        T = sum(rows)
        offs, nts = offs_of(rows), dev32(cand)
        slots = cache.plan(t, offs, nts, total_tokens=T,
                           release=dev32(release) if any(release) else None)
        lengths = [(0 if g else x) + r - c for x, r, c, g in zip(lengths, rows, cand, release)]
        for layer, pg in enumerate(pages):
            q, k, v = silu_rows(T, H, d, 50 * n + layer)
            at = 0
            for b in range(B):
                new = tuple(ref.quantise(x[at:at + rows[b] - cand[b]]) for x in (k, v))
                old = kept[layer][b]
                if old is None or release[b]:
                    kept[layer][b] = tuple(tuple(y.double() for y in x) for x in new)
                else:
                    kept[layer][b] = tuple(tuple(torch.cat([y, z.double()]) for y, z in zip(o, x))
                                           for o, x in zip(old, new))
                at += rows[b]
            qg, kg, vg = (on_gpu(x, True) for x in (q, k, v))
            cache.append(kg, vg, slots, pg, t)
            out = cache.attend(qg, kg, vg, offs, nts, pg, t, contextual_len=ctx, K1=K1, K2=K2,
                               alpha=d ** -0.5, N=64.0, max_new=max(rows))
            want, tol = ref.attend(q, k, v, rows, cand, lengths, kept[layer], K1=K1,
                                   K2e=max(K2, ctx), alpha=d ** -0.5, N=64.0)
            check(out.cpu().double(), want, tol)
        assert t.lengths.tolist() == lengths and cache.get_error(t) == 0


def test_a_captured_step_replays_with_other_lengths():
    """One graph of plan, append and attend on a side stream, replayed with new
    offsets, targets and rows in the same tensors, gives what plain calls give."""
    H, d, ps, B, T = 2, 32, 16, 3, 24
    s = torch.cuda.Stream()
    bufs = [torch.zeros((T, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    offs, nts = dev32([0, 1, 2, 3]), dev32([0, 0, 0])
    ws = torch.empty(4096, dtype=torch.uint8, device=DEV)
    slots = torch.empty(T, dtype=torch.int64, device=DEV)
    out = torch.zeros((T, H, d), dtype=torch.bfloat16, device=DEV)

    def fresh():
        return (cache.allocate_tables(B, 8, 20, page_size=ps, device=DEV),
                torch.zeros((20, H, ps * (d + 8)), dtype=torch.uint8, device=DEV))

    def step(t, pages, slots, out, ws):
        cache.plan(t, offs, nts, total_tokens=T, slots=slots, workspace=ws)
        cache.append(bufs[1], bufs[2], slots, pages, t)
        cache.attend(*bufs, offs, nts, pages, t, contextual_len=2, K1=20, K2=4, alpha=0.2, N=8.0,
                     out=out)

    t1, p1 = fresh()
    t2, p2 = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        step(t1, p1, slots, out, ws)
        graph.capture_end()
    torch.cuda.synchronize()
    for n, (rows, cand) in enumerate([([20, 1, 3], [0, 0, 0]), ([1, 9, 1], [0, 8, 0]),
                                      ([0, 1, 23], [0, 1, 20])]):
        offs.copy_(offs_of(rows))
        nts.copy_(dev32(cand))
        for x, y in zip(bufs, silu_rows(T, H, d, n)):
            x.copy_(y)
        out.fill_(9.0)
        other = torch.full_like(out, 9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        sl = torch.empty_like(slots)
        step(t2, p2, sl, other, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(sl, slots) and torch.equal(t1.buf, t2.buf) and torch.equal(p1, p2)
        assert torch.equal(out, other) and cache.get_error(t1) == 0


def test_python_refusals():
    t, pages, _ = filled([20], 2, 32, 16, 1)
    q, k, v = (x.to(DEV) for x in silu_rows(2, 2, 32, 0))
    offs = offs_of([2])
    kw = dict(contextual_len=0, K1=4, K2=0, alpha=0.1, N=1.0)
    with pytest.raises(TypeError):
        cache.attend(q.float(), k, v, offs, None, pages, t, **kw)
    with pytest.raises(TypeError):
        cache.attend(q, k, v, offs.long(), None, pages, t, **kw)
    with pytest.raises(ValueError):
        cache.attend(q, k, v, offs_of([1, 1]), None, pages, t, **kw)
    with pytest.raises(ValueError):
        cache.attend(q, None, None, offs, dev32([1]), pages, t, **kw)
    with pytest.raises(ValueError):
        cache.attend(q[:, :1], k, v, offs, None, pages, t, **kw)
    with pytest.raises(ValueError):
        cache.attend(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, offs, None, pages, t,
                     **kw)
    with pytest.raises(ValueError):
        cache.append(k, v, torch.zeros(2, dtype=torch.int64, device=DEV), pages[:, :, :-16], t)
    with pytest.raises(TypeError):
        cache.append(k, v, torch.zeros(2, dtype=torch.int32, device=DEV), pages, t)
    with pytest.raises(ValueError):
        cache.append(k[:1], v, torch.zeros(2, dtype=torch.int64, device=DEV), pages, t)
    with pytest.raises(ValueError):
        cache.plan(t, offs, total_tokens=2, slots=torch.empty(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        cache.CacheTables(t.buf[:40], 1, 2, 3, 16)


@pytest.mark.parametrize("H,d,ps,B,most,rows", [(40, 32, 16, 8, 2600, 1), (24, 64, 64, 13, 3000, 2),
                                                (1, 128, 32, 2, 30000, 1), (40, 128, 64, 9, 2900, 1),
                                              (80, 32, 32, 4, 6000, 1)])
def test_long_histories(H, d, ps, B, most, rows):
    """Blocks that walk many key tiles: more than their ring of stages, and more
    than the page ids a warp holds at a time."""
    g = np.random.default_rng(B)
    lengths = g.integers(most // 2, most, size=B).tolist()
    t, host = tables_of(lengths, ps, B)
    pages = torch.full((t.num_pages, H, ps * (d + 8)), 255, dtype=torch.uint8, device=DEV)
    tokens = []
    slots = cache.slot_map(t, offs_of(lengths), total_tokens=sum(lengths))
    gen = torch.Generator(device=DEV).manual_seed(B)
    k, v = (torch.nn.functional.silu(torch.randn((sum(lengths), H, d), generator=gen, device=DEV))
            .bfloat16() for _ in range(2))
    cache.append(k, v, slots, pages, t)
    at = 0
    for n in lengths:
        tokens.append(tuple((c.double(), s, m) for c, s, m in
                            (ref.quantise(x[at:at + n].cpu()) for x in (k, v))))
        at += n
    for K1, bound in ((1 << 20, rows), (1100, rows), (1 << 20, 200)):  # 200: the kernel of many rows
        got, want, tol = run_attend(t, pages, tokens, lengths, [rows] * B, [0] * B, H, d, 3, K1=K1,
                                    K2=100, ctx=0, max_new=bound)
        check(got, want, tol)


# ------------------------------------------------- what a server may also do
KERNELS = [1, 70]  # rows a sequence: either attention kernel


@pytest.mark.parametrize("rows", KERNELS + [9])
@pytest.mark.parametrize("d", [32, 128])
def test_rows_of_any_scale(rows, d):
    """Rows of q from 2^-120 to 2^60, rows of zeros, and one that spans 2^20."""
    H, ps, lengths = 2, 32, [333, 150]

    def edit(q, k, v):
        for t in range(q.shape[0]):
            q[t, t % H] *= 2.0 ** (-120 + 60 * (t % 4))
            if t % 5 == 3:
                q[t, 1] = 0.0
            if t % 7 == 2:
                q[t, 0, ::2] *= 2.0 ** -20
        q[-1, :] *= 2.0 ** 10

    t, pages, tokens = filled(lengths, H, d, ps, 21)
    for cand in ([0, 0], [rows, rows // 2]):
        got, want, tol = run_attend(t, pages, tokens, lengths, [rows, rows], cand, H, d, 2, K1=200,
                                    K2=40, ctx=0, max_new=rows, edit=edit)
        check(got, want, tol)


@pytest.mark.parametrize("rows", [3, 70])
def test_a_row_that_is_not_finite_is_nan_alone(rows):
    H, d, ps, lengths = 2, 64, 16, [200, 260]

    def edit(q, k, v):
        q[1, 0, 5], q[rows + 2, 1, 63] = float("nan"), float("inf")

    t, pages, tokens = filled(lengths, H, d, ps, 22)
    got, want, tol = run_attend(t, pages, tokens, lengths, [rows, rows], [0, 0], H, d, 2, K1=64,
                                K2=0, ctx=0, max_new=rows, edit=edit)
    for at, h in ((1, 0), (rows + 2, 1)):
        assert bool(got[at, h].isnan().all())
        got[at, h], want[at, h], tol[at, h] = 0, 0, 0
    check(got, want, tol)


@pytest.mark.parametrize("rows", KERNELS)
def test_rows_without_a_range(rows):
    """Keys and values that are constant along d have step 0 and are exact."""
    H, d, ps, L = 1, 64, 16, 150
    t, _ = tables_of([L], ps, 3)
    pages = cache.allocate_pages(t.num_pages, H, d, ps, DEV)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((L, H, 1), generator=g).bfloat16().expand(L, H, d).contiguous()
            for _ in range(2))
    cache.append(k.to(DEV), v.to(DEV), cache.slot_map(t, offs_of([L]), total_tokens=L), pages, t)
    tokens = [tuple((c.double(), s, m) for c, s, m in (ref.quantise(k), ref.quantise(v)))]
    assert all(not s.any() for _, s, _ in tokens[0])
    got, want, tol = run_attend(t, pages, tokens, [L], [rows], [0], H, d, 4, K1=1 << 20, K2=0,
                                ctx=0, max_new=rows)
    check(got, want, tol)


@pytest.mark.parametrize("lengths,rows,cand", [([40, 0, 9], [0, 0, 0], [0, 0, 0]),
                                               ([500, 90], [2, 40], [0, 39]),
                                               ([0, 0], [1, 90], [1, 90])])
def test_no_bound_on_the_rows(lengths, rows, cand):
    """max_new left out; steps without a row."""
    t, pages, tokens = filled(lengths, 2, 32, 16, 23)
    got, want, tol = run_attend(t, pages, tokens, lengths, rows, cand, 2, 32, 5, K1=90, K2=10,
                                ctx=3, pad=5)
    check(got, want, tol)


@pytest.mark.parametrize("rows", KERNELS)
def test_sequences_may_share_pages(rows):
    """Several requests that read one user's pages."""
    H, d, ps, L = 2, 128, 64, 700
    t, pages, tokens = filled([L, L, L], H, d, ps, 24)
    t.block_table[1:] = t.block_table[0]
    got, want, tol = run_attend(t, pages, [tokens[0]] * 3, [L] * 3, [rows] * 3, [rows] * 3, H, d,
                                6, K1=1 << 20, K2=0, ctx=0, max_new=rows)
    check(got, want, tol)


@pytest.mark.parametrize("rows", KERNELS)
def test_rows_into_a_wider_tensor(rows):
    """out as a column block: the other columns stay."""
    H, d, ps, lengths = 2, 32, 32, [4000]
    t, pages, _ = filled(lengths, H, d, ps, 25)
    q, k, v = (x.to(DEV) for x in silu_rows(rows, H, d, 1))
    kw = dict(contextual_len=0, K1=1 << 20, K2=0, alpha=0.2, N=50.0, max_new=rows)
    want = cache.attend(q, None, None, offs_of([rows]), None, pages, t, **kw)
    wide = torch.full((rows, 3 * H * d), 4.0, dtype=torch.bfloat16, device=DEV)
    cache.attend(q, None, None, offs_of([rows]), None, pages, t,
                 out=wide[:, H * d:2 * H * d].unflatten(1, (H, d)), **kw)
    assert torch.equal(wide[:, H * d:2 * H * d].unflatten(1, (H, d)), want)
    assert bool((wide[:, :H * d] == 4).all() and (wide[:, 2 * H * d:] == 4).all())


def test_calls_on_a_given_stream():
    """`stream` other than the current one, tensors released right behind the
    calls: what the plain calls give."""
    H, d, ps, lengths, rows = 2, 64, 32, [3000, 20], 70
    t, pages, _ = filled(lengths, H, d, ps, 26)
    t2 = cache.CacheTables(t.buf.clone(), t.B, t.max_pages, t.num_pages, ps)
    p2 = pages.clone()
    q, k, v = (x.to(DEV) for x in silu_rows(2 * rows, H, d, 1))
    offs, nts = offs_of([rows, rows]), dev32([rows, rows - 1])
    kw = dict(contextual_len=0, K1=1 << 20, K2=0, alpha=0.2, N=50.0, max_new=rows)

    def step(t, pages, stream=None):
        slots = cache.plan(t, offs, nts, total_tokens=2 * rows, stream=stream)
        cache.append(k, v, slots, pages, t, stream=stream)
        last = cache.slot_map(t, offs_of([7, 7]), total_tokens=14, stream=stream)
        return (cache.attend(q, k, v, offs, nts, pages, t, stream=stream, **kw),
                *cache.read(last, pages, t, stream=stream))

    want = step(t, pages)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(t2, p2, s)
    assert cache.get_error(t2, s) == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_two_graphs_at_once():
    """Two captured calls over one cache, each with its own workspace, replayed
    on two streams together."""
    H, d, ps, lengths = 1, 128, 64, [6000]
    t, pages, _ = filled(lengths, H, d, ps, 27)
    runs = []
    for rows in KERNELS + [200]:
        q = silu_rows(rows, H, d, rows)[0].to(DEV)
        offs = offs_of([rows])
        kw = dict(contextual_len=0, K1=1 << 20, K2=0, alpha=0.2, N=50.0, max_new=rows)
        want = cache.attend(q, None, None, offs, None, pages, t, **kw)
        torch.cuda.synchronize()
        s, graph, out = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.stream(s):
            graph.capture_begin()
            cache.attend(q, None, None, offs, None, pages, t, out=out, **kw)
            graph.capture_end()
        runs.append((s, graph, out, want, q, offs))
    for _ in range(20):
        for _, _, out, *_ in runs:
            out.zero_()
        torch.cuda.synchronize()
        for s, graph, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, out, want, *_ in runs:
            assert torch.equal(out, want)


@pytest.mark.parametrize("what", ["first", "down", "past", "length", "page", "none"])
def test_slot_map_reports_bad_inputs(what):
    t, _ = tables_of([40, 0, 70], 16, 3)
    offs, T = [0, 30, 30, 50], 50
    if what == "first":
        offs[0] = 1
    if what == "down":
        offs[1] = 20
        offs[2] = 10
    if what == "past":
        offs[3] = 51
    if what == "length":
        t.lengths[2] = 19
    if what == "page":
        t.block_table[2, 3] = -1
    if what == "none":  # no row at all, and offsets that say otherwise
        T = 0
    slots = cache.slot_map(t, dev32(offs), total_tokens=T)
    assert slots.numel() == T and cache.get_error(t) == _abi.ERR_BAD_INPUT
    assert bool(((slots >= -1) & (slots < t.num_pages * 16)).all())


def test_many_blocks_that_report_at_once():
    """Bad slots and pages all over a large call: the places no row names, and the
    rows behind the last sequence, stay as they were, and the next plan starts
    afresh."""
    H, d, ps, B = 3, 64, 16, 40
    lengths = [100 + b for b in range(B)]
    t, pages, tokens = filled(lengths, H, d, ps, 28)
    _, k, v = (x.to(DEV) for x in silu_rows(6000, H, d, 1))
    keep = t.buf.clone()
    for n in range(20):
        before = pages.clone()
        slots = torch.full((6000,), -1, dtype=torch.int64)
        slots[n::3] = t.num_pages * ps + torch.arange(len(slots[n::3]))
        free = int(t.free_pages[0])
        slots[-1] = free * ps + 3  # a good one, in a page nobody has
        cache.append(k, v, slots.to(DEV), pages, t)
        assert cache.get_error(t) == _abi.ERR_BAD_INPUT
        pages[free] = before[free]
        assert torch.equal(pages, before)
        t.buf.copy_(keep)
        for rows in KERNELS:
            t.block_table[n % 3::2, 2] = t.num_pages + 5
            q = k[:B * rows + 9]
            out = torch.full_like(q, 5.0)
            cache.attend(q, None, None, offs_of([rows] * B), None, pages, t, contextual_len=0,
                         K1=1 << 20, K2=0, alpha=0.1, N=9.0, max_new=rows, out=out)
            assert cache.get_error(t) == _abi.ERR_BAD_INPUT
            assert bool((out[B * rows:] == 5).all())
            t.buf.copy_(keep)
    got, want, tol = run_attend(t, pages, tokens, lengths, [1] * B, [0] * B, H, d, 3, K1=1 << 20,
                                K2=0, ctx=0, max_new=1)
    check(got, want, tol)


def test_sizes_beyond_their_fields_are_refused():
    t, pages, _ = filled([20], 2, 32, 16, 1)
    q = silu_rows(2, 2, 32, 0)[0].to(DEV)
    kw = dict(contextual_len=0, K1=4, K2=0, alpha=0.1, N=1.0)
    for name, value in (("K1", 1 << 32), ("K2", 1 << 40), ("contextual_len", 1 << 31),
                        ("max_new", 1 << 33), ("alpha", 1e300), ("N", -1.0)):
        # (a float that fp32 lacks is an infinity, which the library refuses)
        with pytest.raises(SLAError if name in ("alpha", "N") else ValueError):
            cache.attend(q, None, None, offs_of([2]), None, pages, t, **{**kw, name: value})
    for bad in (dict(B=1 << 31), dict(num_pages=1 << 32), dict(page_size=16 + (1 << 32)),
                dict(page_size=48)):
        with pytest.raises(ValueError):
            cache.CacheTables(t.buf, **{**dict(B=1, max_pages=2, num_pages=3, page_size=16), **bad})


def test_long_reads_repeat_themselves():
    """Blocks that go round their ring of key tiles several times, behind others that
    leave other phases in shared memory: every call gives the same bits."""
    H, d, ps = 4, 64, 32
    t, pages, _ = filled([2000, 1500, 900], H, d, ps, 29)
    runs = []
    for rows in (1, 5):
        q = silu_rows(3 * rows, H, d, rows)[0].to(DEV)
        for K1 in (1 << 20, 700):
            args = (q, None, None, offs_of([rows] * 3), None, pages, t)
            kw = dict(contextual_len=0, K1=K1, K2=0, alpha=0.2, N=50.0, max_new=rows)
            runs.append((args, kw, cache.attend(*args, **kw)))
    for _ in range(50):
        for args, kw, want in runs:
            assert torch.equal(cache.attend(*args, **kw), want)
    assert cache.get_error(t) == 0


def test_a_given_stream_leaves_released_memory_alone():
    """Memory released while the current stream still has work on it is not what a call
    on another stream writes, and an output released right behind its use is not written
    again before that use."""
    H, d, ps, rows = 2, 64, 32, 70
    t, pages, _ = filled([3000, 20], H, d, ps, 30)
    q, k, v = (x.to(DEV) for x in silu_rows(2 * rows, H, d, 1))
    offs, nts = offs_of([rows, rows]), dev32([rows, rows - 1])
    last = offs_of([20, 20])
    slots = cache.slot_map(t, last, total_tokens=40)
    kw = dict(contextual_len=0, K1=1 << 20, K2=0, alpha=0.2, N=50.0, max_new=rows)
    calls = [lambda s: cache.attend(q, k, v, offs, nts, pages, t, stream=s, **kw),
             lambda s: cache.read(slots, pages, t, stream=s)[1],
             lambda s: cache.slot_map(t, last, total_tokens=40, stream=s)]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for f, w in zip(calls, want):
        for _ in range(3):
            # as many bytes as the call's output, still to be read here
            held = torch.full_like(w, 7)
            seen = torch.empty_like(held)
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)  # some 10 ms
            seen.copy_(held)
            del held
            got = f(s)
            s.synchronize()
            assert torch.equal(got, w)
            assert bool((seen == 7).all())
            # the other way: an output still to be read here, its memory given back
            torch.cuda._sleep(20_000_000)
            seen.copy_(got)
            del got
            with torch.cuda.stream(s):
                after = torch.full_like(w, 3)
            torch.cuda.synchronize()
            assert torch.equal(seen, w) and bool((after == 3).all())
    assert cache.get_error(t) == 0


@pytest.mark.parametrize("total,most,offs,nts,length,code", [
    (6, 0, [0, 3, 6], [0, 0], 40, _abi.ERR_BAD_INPUT),     # rows where none are announced
    (6, 0, [0, 0, 1], [0, 1], 40, _abi.ERR_BAD_INPUT),
    (6, 0, [0, 0, 0], [0, 0], 40, 0),
    (0, None, [0, 0, 2], [0, 0], 40, _abi.ERR_BAD_INPUT),  # offsets beyond no rows
    (0, None, [0, 1, 0], [0, 0], 40, _abi.ERR_BAD_INPUT),
    (0, None, [0, 0, 0], [0, 1], 40, _abi.ERR_BAD_INPUT),
    (0, None, [0, 0, 0], [0, 0], -1, _abi.ERR_BAD_INPUT),
    (0, 5, [0, 0, 0], [0, 0], 1 << 20, _abi.ERR_BAD_INPUT),
    (0, 5, [0, 0, 0], [0, 0], 40, 0)])
def test_attend_without_rows_still_checks(total, most, offs, nts, length, code):
    H, d, ps = 2, 32, 16
    t, pages, _ = filled([60, 40], H, d, ps, 31)
    t.lengths[1] = length
    q, k, v = (x.to(DEV) for x in silu_rows(total, H, d, 0))
    out = torch.full_like(q, 5.0)
    cache.attend(q, k, v, dev32(offs), dev32(nts), pages, t, contextual_len=0, K1=8, K2=0,
                 alpha=0.1, N=9.0, max_new=most, out=out)
    assert cache.get_error(t) == code and bool((out == 5).all())


def test_attend_without_rows_checks_every_sequence():
    B = 700
    t = cache.allocate_tables(B, 1, 1, page_size=16, device=DEV)
    pages = cache.allocate_pages(1, 1, 32, 16, DEV)
    q = torch.empty((0, 1, 32), dtype=torch.bfloat16, device=DEV)
    offs = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    for bad in (None, 0, 255, 256, 699):
        t.status.zero_()
        t.lengths.zero_()
        if bad is not None:
            t.lengths[bad] = -1
        cache.attend(q, None, None, offs, None, pages, t, contextual_len=0, K1=8, K2=0,
                     alpha=0.1, N=9.0)
        assert cache.get_error(t) == (0 if bad is None else _abi.ERR_BAD_INPUT)


def test_a_set_status_stops_every_call():
    """While the last plan has failed, append, read and either attention kernel, split or
    not, leave everything as it was; slot_map gives no slot; the next plan frees them."""
    H, d, ps = 2, 64, 32
    for lengths in ([3000, 2900], [70, 40]):
        t, pages, _ = filled(lengths, H, d, ps, 32)
        cache.plan(t, offs_of([10 ** 4, 0]), total_tokens=10 ** 4)
        assert cache.get_error(t) != 0
        code, before = cache.get_error(t), (t.buf.clone(), pages.clone())
        slots = cache.slot_map(t, offs_of([5, 5]), total_tokens=10)
        assert bool((slots == -1).all())
        slots = torch.arange(10, device=DEV)
        k, v = (x.to(DEV) for x in silu_rows(10, H, d, 1)[1:])
        cache.append(k, v, slots, pages, t)
        back = [torch.full_like(k, 5.0) for _ in range(2)]
        cache.read(slots, pages, t, k=back[0], v=back[1])
        assert all(bool((x == 5).all()) for x in back)
        for rows, most in ((1, 1), (5, 5), (70, 70), (0, 0)):
            for cand in (None, dev32([rows, rows])):
                q, k, v = (x.to(DEV) for x in silu_rows(2 * rows, H, d, 2))
                out = torch.full_like(q, 5.0)
                cache.attend(q, k, v, offs_of([rows, rows]), cand, pages, t, contextual_len=0,
                             K1=1 << 20, K2=0, alpha=0.1, N=9.0, max_new=most, out=out)
                assert bool((out == 5).all())
        assert cache.get_error(t) == code
        assert torch.equal(t.buf, before[0]) and torch.equal(pages, before[1])
        cache.plan(t, offs_of([1, 0]), total_tokens=1)
        assert cache.get_error(t) == 0


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ahead", [-40, -30, -26])
def test_read_rounds_once(d, ahead):
    """Rows whose s code lies midway between two bf16 numbers (s = 129/2048, codes 3, 6
    and 12) with a minimum below fp32's resolution of it: bf16(m + s code) rounds once."""
    H, ps, T = 2, 16, 40
    g = torch.Generator().manual_seed(d)
    k = torch.rand((T, H, d), generator=g) * (242 / 256)
    k[..., 1] = 242 / 256
    v = k.flip(-1).clone()
    low = torch.where(torch.arange(T) % 2 == 0, -1.0, 1.0) * 2.0 ** ahead
    k[..., 0], v[..., 5] = low[:, None], low[:, None]
    k, v = k.bfloat16(), v.bfloat16()
    t = cache.allocate_tables(1, 1, 4, page_size=ps, device=DEV)
    pages = cache.allocate_pages(4, H, d, ps, DEV)
    slots = torch.randperm(4 * ps, generator=g)[:T].to(DEV)
    cache.append(k.to(DEV), v.to(DEV), slots, pages, t)
    for x, got in zip((k, v), cache.read(slots, pages, t)):
        code, s, m = ref.quantise(x)
        assert bool((s == 129 / 2048).all()) and torch.equal(m, low[:, None].expand(T, H).double())
        exact = m[..., None] + s[..., None] * code  # (fits 53 bits)
        want = ref.bf16_once(exact)
        assert bool((want != exact.float().bfloat16().double()).any())
        assert torch.equal(got.cpu().double(), want)
    assert cache.get_error(t) == 0
