"""The products with 4-bit weights, the norms and rotary positions and the
attention behind shared tokens on the host: refusals (before any GPU call) and
the kernels' resources."""

import ctypes
import re
import subprocess

import pytest

import memory_bound_gemv_f32_amd as lg
from test_code_object import TARGET, _tool
from test_fp8_host import BAD_BATCHES, BAD_CACHES, batch, cache

BAD = lg.GEMV_ERROR_INVALID_VALUE
P = 0x10000
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("fn,size", [(lg.gemv_q4_f32, 4), (lg.gemv_q4_f16, 2), (lg.gemv_q4_bf16, 2)])
def test_product_refusals(fn, size):
    good = dict(Q=P, ldq=151, s=P, lds=3, z=P, ldz=3, group=128, X=P, ldx=301, bias=P, Y=P, dtype=0, ldy=8, M=8, K=301, n=2)

    def call(**kw):
        return fn(*{**good, **kw}.values(), None)
    for kw in (dict(M=-1), dict(K=-1), dict(n=-1), dict(ldq=150), dict(lds=2), dict(ldz=2), dict(ldx=300), dict(ldy=7),
               dict(group=0), dict(group=16), dict(group=48), dict(group=256), dict(group=-32), dict(dtype=3), dict(dtype=-1),
               dict(Q=None), dict(s=None), dict(X=None), dict(Y=None), dict(s=P + 1), dict(X=P + 1), dict(Y=P + 1),
               dict(Y=P + 2), dict(Y=P + 1, dtype=1), dict(bias=P + 2), dict(group=32)):
        assert call(**kw) == BAD, kw
    assert call(M=0, Y=None) == 0 and call(n=0, Y=None) == 0


def part(**kw):
    a = dict(x=P, ldx=256, y=P, ldy=256, heads=2, y_dtype=0, weight=P)
    a.update(kw)
    return lg.RotaryPartStruct(*a.values())


@pytest.mark.parametrize("fn,size", [(lg.gemv_rotary_f32, 4), (lg.gemv_rotary_f16, 2), (lg.gemv_rotary_bf16, 2)])
def test_rotary_refusals(fn, size):
    def call(parts=None, b=None, **kw):
        a = dict(count=2, dim=128, rows=5, frequency=P, pairs=64, interleaved=0, magnitude=1.0, eps=1e-6)
        a.update(kw)
        array = (lg.RotaryPartStruct * 8)(*(parts or [part(), part()]))
        return fn(array, *a.values(), ctypes.byref(b or batch()), None)
    inf, nan = float("inf"), float("nan")
    for kw in (dict(count=0), dict(count=5), dict(count=-1), dict(dim=0), dict(dim=127), dict(dim=514), dict(dim=-2),
               dict(dim=130), dict(rows=-1), dict(pairs=-1), dict(pairs=65), dict(frequency=None), dict(frequency=P + 2),
               dict(interleaved=2), dict(interleaved=-1), dict(magnitude=inf), dict(magnitude=nan), dict(eps=-1e-9),
               dict(eps=inf), dict(eps=nan)):
        assert call(**kw) == BAD, kw
    for kw in (dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 2), dict(weight=P + 2), dict(ldx=255), dict(ldy=255),
               dict(heads=-1), dict(y_dtype=3), dict(y_dtype=-1), dict(heads=MOST, ldx=MOST, ldy=MOST)):
        assert call(parts=[part(), part(**kw)]) == BAD, kw
    for kw in (dict(sequences=-1), dict(seq_lens=None), dict(seq_lens=P + 2), dict(starts=P + 2), dict(starts=None)):
        assert call(b=batch(**kw)) == BAD, kw
    # more rows than a launch holds
    assert call(rows=(1 << 25) + 1) == BAD
    array = (lg.RotaryPartStruct * 1)(part())
    assert fn(None, 1, 128, 5, P, 64, 0, 1.0, 1e-6, ctypes.byref(batch()), None) == BAD
    assert fn(array, 1, 128, 5, P, 64, 0, 1.0, 1e-6, None, None) == BAD
    # nothing to do
    assert call(rows=0) == 0 and call(b=batch(sequences=0)) == 0
    assert call(parts=[part(heads=0), part(heads=0, x=None, y=None)]) == 0


@pytest.mark.parametrize("fn", [lg.gemv_kv_attend_shared_f16, lg.gemv_kv_attend_shared_bf16])
def test_shared_refusals(fn):
    def call(c=None, b=None, Q=P, ldq=1024, O=P, ldo=1024, heads=8, rows=5, scale=0.1, window=0, sinks=0, shared=100,
             ws=P, wsb=1 << 40):
        return fn(ctypes.byref(c or cache()), Q, ldq, O, ldo, heads, rows, ctypes.byref(b or batch()), scale, window,
                  sinks, shared, ws, wsb, None)
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == BAD, kw
    inf, nan = float("inf"), float("nan")
    for kw in (dict(Q=None), dict(O=None), dict(Q=P + 1), dict(O=P + 1), dict(ldq=1023), dict(ldo=1023), dict(heads=7),
               dict(heads=0), dict(rows=-1), dict(scale=inf), dict(scale=nan), dict(window=-1), dict(sinks=-1),
               dict(shared=-1), dict(heads=1 << 20, ldq=1 << 30, ldo=1 << 30, rows=1 << 12)):
        assert call(**kw) == BAD, kw
    # results over shared tokens are joined: the call needs its workspace
    n = ctypes.c_size_t()
    size = lg.gemv_kv_attend_shared_workspace_size
    assert size(8, 2, 128, 2, 2, 1, 1000, 64, 0, 0, 60000, ctypes.byref(n)) == 0 and n.value > 0
    wide = dict(b=batch(table_width=1000, table_pitch=1000, starts=None), rows=2, shared=60000)
    assert call(**wide, ws=None) == BAD and call(**wide, wsb=n.value - 1) == BAD and call(**wide, ws=P + 8) == BAD
    assert call(rows=0) == 0


def test_shared_workspace_size():
    n, plain = ctypes.c_size_t(7), ctypes.c_size_t(7)
    f = lg.gemv_kv_attend_shared_workspace_size
    good = dict(q_heads=8, heads=2, dim=128, rows=3, sequences=3, one_each=1, table_width=100, page_size=64, window=0,
                sinks=0, shared=1000)
    assert f(*good.values(), ctypes.byref(n)) == 0 and n.value > 0 and n.value % 16 == 0
    for bad in (dict(q_heads=7), dict(q_heads=0), dict(heads=0), dict(dim=100), dict(rows=-1), dict(sequences=-1),
                dict(rows=2), dict(table_width=-1), dict(page_size=8), dict(window=-1), dict(sinks=-1), dict(shared=-1),
                dict(heads=65536, q_heads=65536), dict(one_each=0, sequences=MOST)):
        assert f(*{**good, **bad}.values(), ctypes.byref(n)) == BAD, bad
    assert f(*good.values(), None) == BAD
    # nothing shared: what the call without it needs
    for none in (dict(shared=0), dict(shared=63), dict(rows=1, sequences=1)):
        a = {**good, **none}
        assert f(*a.values(), ctypes.byref(n)) == 0
        a.pop("shared")
        assert lg.gemv_kv_attend_workspace_size(*a.values(), ctypes.byref(plain)) == 0 and plain.value == n.value
    # bounded, however much is shared
    for width in (1, 10, 1000, 100000, 1 << 25):
        for shared in (64, 1000, 1 << 20, MOST):
            for rows in (2, 64, 300):
                a = {**good, "table_width": width, "shared": shared, "rows": rows, "sequences": rows}
                assert f(*a.values(), ctypes.byref(n)) == 0 and n.value < 1 << 30, a


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Metadata of the kernels of the 4-bit products and rotary positions."""
    tmp = tmp_path_factory.mktemp("objects")
    fat = tmp / "fatbin"
    subprocess.run([_tool("llvm-objcopy"), f"--dump-section=.hip_fatbin={fat}", str(lg.LIBRARY), str(tmp / "rest")],
                   check=True, capture_output=True)
    data = fat.read_bytes()
    at = [m.start() for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data)]
    found = {}
    for i, a in enumerate(at):
        (tmp / "bundle").write_bytes(data[a:at[i + 1] if i + 1 < len(at) else len(data)])
        subprocess.run([_tool("clang-offload-bundler"), "--unbundle", "--type=o", f"--targets={TARGET}",
                        f"--input={tmp / 'bundle'}", f"--output={tmp / 'object'}"], check=True, capture_output=True)
        notes = subprocess.run([_tool("llvm-readelf"), "--notes", str(tmp / "object")], check=True,
                               capture_output=True, text=True).stdout
        for entry in re.split(r"\n  - (?=\.)", notes)[1:]:
            fields = dict(re.findall(r"\.(\w+):[ ]+(\S+)", entry))
            name = fields.get("symbol", "")
            if "q4dev" in name or "rotarydev" in name:
                found[name] = fields
    return found


def test_kernels_use_no_scratch(kernels):
    for family in ("q4_few", "rotary"):
        assert any(family in n for n in kernels), family
    for name, f in kernels.items():
        assert f["private_segment_fixed_size"] == "0" and f["vgpr_spill_count"] == "0", name
        assert f["uses_dynamic_stack"] == "false" and f["wavefront_size"] == "64", name
        waves = max(1, -(-int(f["max_flat_workgroup_size"]) // 256))
        assert int(f["vgpr_count"]) <= 512 // waves, name
        assert int(f["group_segment_fixed_size"]) <= 160 * 1024, name


def test_every_family_is_built(kernels):
    """... and so held to the limits above."""
    for family in ("q4_short", "q4_few", "q4_tile", "q4_wide", "rotary"):
        assert any(family in n for n in kernels), family
