"""The paged 4-bit history cache without a GPU: the 64-bit forms the GPU tests
compare with, the masks and key tiles, and the refusals of the C ABI and the
binding."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import cache_ref as ref
from sparse_hstu_attention_b200 import _abi, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every case below fails a host check first


@pytest.fixture(scope="module")
def lib():
    from sparse_hstu_attention_b200 import build
    build.build()
    return _abi.load()


def test_masks_and_key_tiles_are_exact(tmp_path):
    exe = str(tmp_path / "cache_enum_check")
    subprocess.check_call(["/usr/local/cuda/bin/nvcc", "-std=c++17", "-O2",
                           "-Wno-deprecated-gpu-targets", "-x", "cu",
                           os.path.join(ROOT, "tests", "cache_enum_check.cu"), "-o", exe])
    r = subprocess.run([exe, "1500"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("OK"), r.stdout + r.stderr


@pytest.mark.parametrize("H,d,ps", [(1, 32, 16), (3, 64, 32), (2, 128, 64)])
def test_layout_round_trip(H, d, ps):
    """Every byte of a page belongs to one token's codes or pairs, and a packed
    row reads back as m + s code."""
    kb, ks, vb, vs, kp, vp = ref.offsets(H, d, ps)
    used = np.concatenate([(kb * 2 + ks // 4).ravel(), (vb * 2 + vs // 4).ravel()] +
                          [(2 * (p + i) + z).ravel() for p in (kp, vp) for i in range(4)
                           for z in (0, 1)])
    assert np.array_equal(np.sort(used), np.arange(2 * H * ps * (d + 8)))
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn((2 * ps, H, d), generator=g).bfloat16() for _ in range(2))
    pages = torch.randint(0, 256, (2, H, ps * (d + 8)), generator=g, dtype=torch.uint8)
    slots = torch.randperm(2 * ps, generator=g)
    pages = ref.pack(pages, ps, slots, k, v)
    K, V = ref.unpack(pages, ps, d)
    assert torch.equal(K.reshape(-1, H, d)[slots], ref.values(k))
    assert torch.equal(V.reshape(-1, H, d)[slots], ref.values(v))


def test_quantisation_error_is_half_a_step():
    """|x - (m + s code)| <= s/2, plus what rounding s to bf16 leaves at the top
    code (15 steps of half a bf16 ulp each) and a few fp32 roundings."""
    g = torch.Generator().manual_seed(1)
    x = torch.nn.functional.silu(torch.randn((500, 128), generator=g) * 2).bfloat16()
    c, s, m = ref.quantise(x)
    assert c.min() == 0 and c.max() == 15
    err = (x.double() - ref.values(x)).abs()
    assert (err <= s[:, None] * (0.5 + 15 * 2.0 ** -8 + 1e-5)).all()
    flat = torch.full((2, 32), 3.5).bfloat16()
    assert torch.equal(ref.values(flat), flat.double())
    odd = torch.zeros((2, 32)).bfloat16()
    odd[0, 3], odd[1, 5] = float("nan"), float("inf")
    assert torch.isnan(ref.values(odd)).all()


def test_bf16_once_rounds_to_the_nearest():
    """On fp32 numbers it is torch's rounding (subnormal ones too); on numbers next to a
    midpoint it goes to the side they are on."""
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-2 ** 31, 2 ** 31, (20000,), generator=g).int().view(torch.float32)
    x = x[x.abs() < 3e38]
    assert torch.equal(ref.bf16_once(x), x.bfloat16().double())
    assert (x.abs() < 2.0 ** -126).any()
    mid = 1 + 2.0 ** -8
    x = torch.tensor([mid, mid + 2.0 ** -40, mid - 2.0 ** -40, -mid - 2.0 ** -40],
                     dtype=torch.float64)
    assert ref.bf16_once(x).tolist() == [1, 1 + 2.0 ** -7, 1, -1 - 2.0 ** -7]


def _tables(**kw):
    t = _abi.CacheTablesC(4, 8, 32, 64, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _rows(**kw):
    r = _abi.CacheRows(4, 128, 10, FAKE, FAKE, 4 * 64 * 136, FAKE, FAKE, 512, 512)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _attend(**kw):
    p = _abi.CacheAttendParams(4, 128, 10, 10, FAKE, FAKE, 0, 8, 4, 0.1, 10.0, FAKE, FAKE, FAKE,
                               512, 512, 512, FAKE, 4 * 64 * 136, FAKE, 512)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD_TABLES = [("B", 0, _abi.ERR_INVALID_ARG), ("max_pages", 0, _abi.ERR_INVALID_ARG),
              ("max_pages", (1 << 19) + 1, _abi.ERR_UNSUPPORTED),
              ("num_pages", 0, _abi.ERR_INVALID_ARG), ("page_size", 48, _abi.ERR_UNSUPPORTED),
              ("page_size", 128, _abi.ERR_UNSUPPORTED), ("status", None, _abi.ERR_INVALID_ARG),
              ("lengths", FAKE + 2, _abi.ERR_INVALID_ARG),
              ("free_pages", None, _abi.ERR_INVALID_ARG),
              ("block_table", None, _abi.ERR_INVALID_ARG)]


@pytest.mark.parametrize("field,value,code", BAD_TABLES)
def test_bad_tables_are_refused(lib, field, value, code):
    t = _tables(**{field: value})
    assert lib.hstu_cache_plan(t, FAKE, None, None, 10, FAKE, FAKE, 1 << 20, None) == code
    assert lib.hstu_cache_slot_map(t, FAKE, 10, FAKE, None) == code
    assert lib.hstu_cache_append(t, _rows(), None) == code
    assert lib.hstu_cache_read(t, _rows(), None) == code
    assert lib.hstu_cache_attend(t, _attend(), FAKE, 1 << 30, None) == code
    assert lib.hstu_cache_attend_workspace_bytes(t, _attend()) == 0


def test_plan_refusals(lib):
    t = _tables()
    f, bytes_of = lib.hstu_cache_plan, lib.hstu_cache_plan_workspace_bytes
    assert bytes_of(0, 10) == 0 and bytes_of(4, -1) == 0
    assert bytes_of(4, 10) == 0  # a small step keeps its sums on chip
    T = 100_000
    need = bytes_of(4, T)
    assert need >= 256 and need % 256 == 0 and bytes_of(5000, 1) > 0
    assert f(None, FAKE, None, None, T, FAKE, FAKE, need, None) == _abi.ERR_INVALID_ARG
    assert f(t, None, None, None, T, FAKE, FAKE, need, None) == _abi.ERR_INVALID_ARG
    assert f(t, FAKE, None, None, -1, FAKE, FAKE, need, None) == _abi.ERR_INVALID_ARG
    assert f(t, FAKE, None, None, T, FAKE + 4, FAKE, need, None) == _abi.ERR_INVALID_ARG
    assert f(t, FAKE, None, None, 1 << 31, FAKE, FAKE, need, None) == _abi.ERR_UNSUPPORTED
    assert f(t, FAKE, None, None, T, FAKE, None, need, None) == _abi.ERR_WORKSPACE
    assert f(t, FAKE, None, None, T, FAKE, FAKE + 128, need, None) == _abi.ERR_WORKSPACE
    assert f(t, FAKE, None, None, T, FAKE, FAKE, need - 1, None) == _abi.ERR_WORKSPACE


@pytest.mark.parametrize("field,value,code", [
    ("H", 0, _abi.ERR_INVALID_ARG), ("d", 96, _abi.ERR_UNSUPPORTED),
    ("T", -1, _abi.ERR_INVALID_ARG), ("T", 1 << 31, _abi.ERR_UNSUPPORTED),
    ("slots", None, _abi.ERR_INVALID_ARG), ("pages", FAKE + 8, _abi.ERR_INVALID_ARG),
    ("page_stride", 4 * 64 * 136 - 16, _abi.ERR_INVALID_ARG),
    ("page_stride", 4 * 64 * 136 + 8, _abi.ERR_INVALID_ARG),
    ("k", None, _abi.ERR_INVALID_ARG), ("v", FAKE + 2, _abi.ERR_INVALID_ARG),
    ("k_row_stride", 504, _abi.ERR_INVALID_ARG), ("v_row_stride", 516, _abi.ERR_INVALID_ARG)])
def test_rows_refusals(lib, field, value, code):
    assert lib.hstu_cache_append(_tables(), _rows(**{field: value}), None) == code
    assert lib.hstu_cache_read(_tables(), _rows(**{field: value}), None) == code


@pytest.mark.parametrize("field,value,code", [
    ("H", 0, _abi.ERR_INVALID_ARG), ("d", 16, _abi.ERR_UNSUPPORTED),
    ("max_new", -1, _abi.ERR_INVALID_ARG), ("K1", -1, _abi.ERR_INVALID_ARG),
    ("K2", -1, _abi.ERR_INVALID_ARG), ("contextual_len", -1, _abi.ERR_INVALID_ARG),
    ("N", 0.0, _abi.ERR_INVALID_ARG), ("alpha", float("nan"), _abi.ERR_INVALID_ARG),
    ("seq_offsets", None, _abi.ERR_INVALID_ARG), ("q", None, _abi.ERR_INVALID_ARG),
    ("k", None, _abi.ERR_INVALID_ARG), ("v", FAKE + 8, _abi.ERR_INVALID_ARG),
    ("out", None, _abi.ERR_INVALID_ARG), ("q_row_stride", 256, _abi.ERR_INVALID_ARG),
    ("out_row_stride", 513, _abi.ERR_INVALID_ARG), ("pages", None, _abi.ERR_INVALID_ARG),
    ("total_tokens", 1 << 31, _abi.ERR_UNSUPPORTED)])
def test_attend_refusals(lib, field, value, code):
    p = _attend(**{field: value})
    assert lib.hstu_cache_attend(_tables(), p, FAKE, 1 << 30, None) == code
    assert lib.hstu_cache_attend_workspace_bytes(_tables(), p) == 0


def test_attend_workspace_refusals(lib):
    # two sequences of one row and long histories: the keys are split over blocks
    p = _attend(total_tokens=4, max_new=1, K1=1 << 20)
    t = _tables(max_pages=4096)
    need = lib.hstu_cache_attend_workspace_bytes(t, p)
    assert need >= 256 and need % 256 == 0
    f = lib.hstu_cache_attend
    assert f(t, p, None, need, None) == _abi.ERR_WORKSPACE
    assert f(t, p, FAKE + 64, need, None) == _abi.ERR_WORKSPACE
    assert f(t, p, FAKE, need - 1, None) == _abi.ERR_WORKSPACE


def test_binding_structs_match_the_header(tmp_path):
    """The binding's ctypes structs have the C compiler's size and offsets."""
    for py, c in ((_abi.CacheTablesC, "hstu_cache_tables"), (_abi.CacheRows, "hstu_cache_rows"),
                  (_abi.CacheAttendParams, "hstu_cache_attend_params")):
        names = [f[0] for f in py._fields_]
        src = tmp_path / "layout.c"
        src.write_text("\n".join(
            ['#include <stdio.h>', '#include <stddef.h>', '#include "hstu_cache.h"',
             'int main(void) {', f'printf("%zu\\n", sizeof({c}));'] +
            [f'printf("%zu\\n", offsetof({c}, {f}));' for f in names] + ['return 0; }']))
        exe = tmp_path / "layout"
        subprocess.run(["gcc", "-std=c99", "-I", _abi.INCLUDE_DIR, str(src), "-o", str(exe)],
                       check=True)
        got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                              text=True).stdout.split()]
        assert got == [ctypes.sizeof(py)] + [getattr(py, n).offset for n in names]


def test_tables_refuse_wrong_buffers():
    n = cache.CacheTables.words(3, 5, 7)
    assert n == 64 + 64 + 64 + 15
    with pytest.raises(TypeError):
        cache.CacheTables(torch.zeros(n, dtype=torch.int32), 3, 5, 7, 64)  # not on a GPU


def test_packed_arguments_have_the_structs_layout():
    """CACHE_ROWS and CACHE_ATTEND place every field where the ctypes structs do."""
    for layout, struct_ in ((_abi.CACHE_ROWS, _abi.CacheRows),
                            (_abi.CACHE_ATTEND, _abi.CacheAttendParams)):
        values = [0.5 * i if t is ctypes.c_float else 3 * i + 1
                  for i, (_, t) in enumerate(struct_._fields_)]
        s = struct_.from_buffer_copy(layout.pack(*values))
        assert ctypes.sizeof(struct_) == layout.size
        assert [getattr(s, n) for n, _ in struct_._fields_] == values


def test_arguments_beyond_their_fields_are_refused():
    """A window of 2^40 is refused, not taken modulo 2^32."""
    ok = [4, 128, 10, 10, FAKE, 0, 0, 8, 4, 0.1, 10.0, FAKE, FAKE, FAKE, 512, 512, 512, FAKE, 64,
          FAKE, 512]
    assert len(cache._pack(_abi.CACHE_ATTEND, *ok)) == ctypes.sizeof(_abi.CacheAttendParams)
    for at, value in ((3, 1 << 31), (6, -1 << 40), (7, 1 << 32), (8, 1 << 40), (9, 10 ** 400)):
        with pytest.raises(ValueError):
            cache._pack(_abi.CACHE_ATTEND, *ok[:at], value, *ok[at + 1:])


@pytest.mark.parametrize("max_new,total", [(1, 10), (16, 1 << 20), (1 << 20, 1 << 20),
                                           ((1 << 31) - 1, (1 << 31) - 1)])
def test_more_blocks_than_a_grid_are_refused(lib, max_new, total):
    t = _tables(B=1 << 30)
    p = _attend(max_new=max_new, total_tokens=total, H=65535, page_stride=65535 * 64 * 136,
                **{k: 65535 * 128 for k in ("q_row_stride", "k_row_stride", "v_row_stride",
                                            "out_row_stride")})
    assert lib.hstu_cache_attend(t, p, FAKE, 1 << 60, None) == _abi.ERR_UNSUPPORTED
    assert lib.hstu_cache_attend(_tables(B=(1 << 30) + 1), p, FAKE, 1 << 60,
                                 None) == _abi.ERR_UNSUPPORTED


def test_the_ring_of_key_tiles_never_runs_ahead(tmp_path):
    """No order of the warps and copies lets a warp take a stage before its tile, whatever
    shared memory held; with the stages' words left as they were, some do."""
    exe = str(tmp_path / "cache_ring_check")
    subprocess.check_call(["/usr/local/cuda/bin/nvcc", "-std=c++17", "-O2",
                           "-Wno-deprecated-gpu-targets", "-x", "cu",
                           os.path.join(ROOT, "tests", "cache_ring_check.cu"), "-o", exe])
    for args in (["3000"], ["3000", "keep"]):
        r = subprocess.run([exe, *args], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.startswith("OK"), r.stdout + r.stderr


def test_what_a_call_allocates_comes_from_its_stream(monkeypatch):
    """With a stream given, outputs and scratch are allocated with that stream current,
    and only outputs are kept for the caller's; without one, nothing is switched."""
    now, made, kept = ["caller's"], [], []

    class Current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            now.append(self.stream)

        def __exit__(self, *_):
            now.pop()

    empty = torch.empty

    def recorded_empty(*a, **kw):
        made.append(now[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: now[-1])
    monkeypatch.setattr(torch, "empty", recorded_empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.dtype, s)),
                        raising=False)
    cpu = torch.device("cpu")
    for stream, where in ((None, "caller's"), ("given", "given")):
        made.clear(), kept.clear()
        assert cache._slots_out(None, 5, cpu, stream).shape == (5,)
        assert cache._workspace(None, 256, cpu, stream).dtype == torch.uint8
        assert made == [where] * 2
        assert kept == ([] if stream is None else [(torch.int64, "caller's")])


def test_bytes_in_shared_memory_state_their_alignment():
    """A byte array in shared memory has an alignment of one unless it says otherwise,
    and the kernels read theirs as words.  (Those of a launch's own size are aligned by
    the kernel, from their address.)"""
    found = 0
    for name in sorted(os.listdir(os.path.join(_abi.PKG, "csrc"))):
        text = open(os.path.join(_abi.PKG, "csrc", name)).read()
        for m in re.finditer(r"(extern )?__shared__ ([^;]*\b(?:u?int8_t|(?:unsigned )?char) [^;]*);",
                             text):
            found += 1
            assert m[1] or re.match(r"__align__\((4|8|16|128)\) ", m[2]), (name, m[0])
    assert found > 5
