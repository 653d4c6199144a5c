"""The 8-bit operators on the host: refusals (before any GPU call) and the
code objects of every source."""

import ctypes
import re
import subprocess

import pytest

import memory_bound_gemv_f32_amd as lg
from test_code_object import TARGET, _tool

BAD = lg.GEMV_ERROR_INVALID_VALUE
P = 0x10000


@pytest.mark.parametrize("fn,size", [(lg.gemv_fp8_quantise_f32, 4), (lg.gemv_fp8_quantise_f16, 2),
                                     (lg.gemv_fp8_quantise_bf16, 2)])
def test_quantise_refusals(fn, size):
    good = dict(X=P, ldx=300, Q=P, ldq=300, s=P, lds=3, rows=4, K=300, block=1)
    def call(**kw):
        a = {**good, **kw}
        return fn(a["X"], a["ldx"], a["Q"], a["ldq"], a["s"], a["lds"], a["rows"], a["K"], a["block"], None)
    for kw in (dict(rows=-1), dict(K=-1), dict(ldx=299), dict(ldq=299), dict(lds=2), dict(block=0), dict(block=64),
               dict(X=None), dict(Q=None), dict(s=None), dict(X=P + 1), dict(s=P + 2),
               dict(block=128, rows=65536 * 128)):
        assert call(**kw) == BAD, kw
    assert call(rows=0) == 0 and call(K=0, X=None, Q=None, s=None) == 0


@pytest.mark.parametrize("fn,size", [(lg.gemv_fp8_f32, 4), (lg.gemv_fp8_f16, 2), (lg.gemv_fp8_bf16, 2)])
def test_product_refusals(fn, size):
    good = dict(W=P, ldw=300, ws=P, ldws=3, X=P, ldx=300, xs=P, ldxs=3, bias=None, Y=P, ldy=8, M=8, K=300, n=2)
    def call(**kw):
        a = {**good, **kw}
        return fn(a["W"], a["ldw"], a["ws"], a["ldws"], a["X"], a["ldx"], a["xs"], a["ldxs"], a["bias"], a["Y"],
                  a["ldy"], a["M"], a["K"], a["n"], None)
    for kw in (dict(M=-1), dict(K=-1), dict(n=-1), dict(ldw=299), dict(ldx=299), dict(ldy=7), dict(ldws=2),
               dict(ldxs=2), dict(W=None), dict(X=None), dict(ws=None), dict(xs=None), dict(Y=None), dict(Y=P + 1),
               dict(ws=P + 1), dict(xs=P + 2), dict(bias=P + 1)):
        assert call(**kw) == BAD, kw
    assert call(M=0, Y=None) == 0 and call(n=0, Y=None) == 0


def cache(**kw):
    a = dict(format=lg.KV_INT8, pages=4, heads=2, page_size=64, dim=128, k=P, v=P, k_scale=P, v_scale=P)
    a.update(kw)
    return lg.KvCacheStruct(*a.values())


def batch(**kw):
    a = dict(sequences=2, table=P, table_pitch=3, table_width=3, seq_lens=P, starts=P)
    a.update(kw)
    return lg.KvBatchStruct(*a.values())


BAD_CACHES = [dict(format=2), dict(format=-1), dict(pages=0), dict(heads=0), dict(heads=65536), dict(page_size=8),
              dict(page_size=48), dict(page_size=512), dict(dim=96), dict(dim=512), dict(k=None), dict(v=None),
              dict(k_scale=None), dict(v_scale=None), dict(k=P + 8), dict(v=P + 4), dict(k_scale=P + 1)]
BAD_BATCHES = [dict(sequences=-1), dict(table=None), dict(table_width=-1), dict(table_pitch=2), dict(seq_lens=None),
               dict(seq_lens=P + 2), dict(table=P + 1), dict(starts=P + 2), dict(starts=None)]


@pytest.mark.parametrize("fn,size", [(lg.gemv_kv_append_f32, 4), (lg.gemv_kv_append_f16, 2),
                                     (lg.gemv_kv_append_bf16, 2)])
def test_append_refusals(fn, size):
    def call(c=None, b=None, K=P, ldk=256, V=P, ldv=256, rows=5):
        return fn(ctypes.byref(c or cache()), K, ldk, V, ldv, rows, ctypes.byref(b or batch()), None)
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == BAD, kw
    for kw in (dict(K=None), dict(V=None), dict(K=P + 1), dict(V=P + 1), dict(ldk=255), dict(ldv=255), dict(rows=-1)):
        assert call(**kw) == BAD, kw
    assert fn(None, P, 256, P, 256, 5, ctypes.byref(batch()), None) == BAD
    assert fn(ctypes.byref(cache()), P, 256, P, 256, 5, None, None) == BAD
    assert call(rows=0) == 0
    assert call(b=batch(sequences=0), rows=5) == 0


@pytest.mark.parametrize("fn", [lg.gemv_kv_attend_f16, lg.gemv_kv_attend_bf16])
def test_attend_refusals(fn):
    def call(c=None, b=None, Q=P, ldq=1024, O=P, ldo=1024, heads=8, rows=5, scale=0.1, window=0, sinks=0, ws=P,
             wsb=1 << 40):
        return fn(ctypes.byref(c or cache()), Q, ldq, O, ldo, heads, rows, ctypes.byref(b or batch()), scale, window,
                  sinks, ws, wsb, None)
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == BAD, kw
    inf, nan = float("inf"), float("nan")
    for kw in (dict(Q=None), dict(O=None), dict(Q=P + 1), dict(O=P + 1), dict(ldq=1023), dict(ldo=1023),
               dict(heads=7), dict(heads=0), dict(rows=-1), dict(scale=inf), dict(scale=-inf), dict(scale=nan),
               dict(window=-1), dict(sinks=-1), dict(heads=1 << 20, ldq=1 << 30, ldo=1 << 30, rows=1 << 12)):
        assert call(**kw) == BAD, kw
    # a batch that is split over its tokens needs its workspace
    n = ctypes.c_size_t()
    assert lg.gemv_kv_attend_workspace_size(8, 2, 128, 2, 2, 1, 1000, 64, 0, 0, ctypes.byref(n)) == 0 and n.value > 0
    wide = dict(b=batch(table_width=1000, table_pitch=1000, starts=None), rows=2)
    assert call(**wide, ws=None) == BAD and call(**wide, wsb=n.value - 1) == BAD and call(**wide, ws=P + 8) == BAD
    assert call(rows=0) == 0


def test_workspace_size():
    n = ctypes.c_size_t(7)
    f = lg.gemv_kv_attend_workspace_size
    good = dict(q_heads=8, heads=2, dim=128, rows=1, sequences=1, one_each=1, table_width=100, page_size=64, window=0,
                sinks=0)
    assert f(*good.values(), ctypes.byref(n)) == 0 and n.value > 0 and n.value % 16 == 0
    for bad in (dict(q_heads=7), dict(q_heads=0), dict(heads=0), dict(dim=100), dict(rows=-1), dict(sequences=-1),
                dict(rows=2), dict(table_width=-1), dict(page_size=8), dict(window=-1), dict(sinks=-1)):
        assert f(*{**good, **bad}.values(), ctypes.byref(n)) == BAD, bad
    assert f(*good.values(), None) == BAD
    for none in (dict(rows=0, sequences=0), dict(table_width=0), dict(table_width=8), dict(window=100)):
        assert f(*{**good, **none}.values(), ctypes.byref(n)) == 0 and n.value == 0, none
    # a longer table never needs less, and the workspace stays bounded
    last = 0
    for width in (1, 10, 100, 1000, 10000, 1 << 25):
        assert f(*{**good, "table_width": width}.values(), ctypes.byref(n)) == 0 and n.value >= last
        last = n.value
    assert last < 1 << 30


def test_workspace_size_refuses_what_a_call_refuses():
    n = ctypes.c_size_t(7)
    good = dict(q_heads=8, heads=2, dim=128, rows=1, sequences=1, one_each=0, table_width=100, page_size=64, window=0,
                sinks=0)
    def size(**kw):
        return lg.gemv_kv_attend_workspace_size(*{**good, **kw}.values(), ctypes.byref(n))
    for page in (16, 32, 64, 128, 256):
        assert size(page_size=page) == 0
    for bad in (dict(page_size=48), dict(page_size=512), dict(page_size=24), dict(heads=65536, q_heads=65536),
                dict(rows=1 << 29), dict(rows=1 << 20, q_heads=1 << 12)):
        assert size(**bad) == BAD, bad
    # more workgroups than a launch holds: refused by both, whatever the products of the sizes
    most = 2 ** 31 - 1
    for many in (dict(sequences=most), dict(sequences=most, heads=65535, q_heads=65535),
                 dict(sequences=most, heads=65535, q_heads=65535, table_width=most, page_size=256),
                 dict(sequences=1 << 24, heads=2), dict(sequences=1 << 24, heads=2, table_width=1)):
        assert size(**many) == BAD, many
        a = {**good, **many}
        ld = a["q_heads"] * 128
        call = lg.gemv_kv_attend_f16(
            ctypes.byref(cache(heads=a["heads"], page_size=a["page_size"])), P, ld, P, ld, a["q_heads"], 1,
            ctypes.byref(batch(sequences=a["sequences"], table_width=a["table_width"], table_pitch=a["table_width"])),
            0.1, 0, 0, P, 1 << 62, None)
        assert call == BAD, many
    for many in (dict(sequences=1 << 20, heads=3, q_heads=3), dict(sequences=1 << 20, rows=1 << 25)):
        assert size(**many) == 0, many


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Metadata of every kernel of the 8-bit operators in the library: each
    source brings a code object of its own."""
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
            if "fp8dev" in name or "kvdev" in name:
                found[name] = fields
    return found


def test_kernels_use_no_scratch(kernels):
    for family in ("fp8_quantise_rows", "fp8_quantise_tile", "fp8_few", "fp8_tile", "fp8_split", "kv_append", "kv_attend", "kv_join"):
        assert any(family in n for n in kernels), family
    for name, f in kernels.items():
        assert f["private_segment_fixed_size"] == "0" and f["vgpr_spill_count"] == "0", name
        assert f["uses_dynamic_stack"] == "false" and f["wavefront_size"] == "64", name
        waves = max(1, -(-int(f["max_flat_workgroup_size"]) // 256))
        assert int(f["vgpr_count"]) <= 512 // waves, name
        assert int(f["group_segment_fixed_size"]) <= 160 * 1024, name


def test_assembly_declares_what_it_writes():
    """Every statement that writes m0 names it, and memory, to the compiler."""
    found = 0
    for source in sorted(lg.LIBRARY.parent.joinpath("csrc").iterdir()):
        for statement in re.findall(r"asm volatile\((.*?)\);", source.read_text(), re.S):
            text, *operands = statement.split("\n")
            if re.search(r"s_mov_b32 m0", text):
                found += 1
                clobbers = " ".join(operands).rsplit(":", 1)[1]
                assert '"m0"' in clobbers and '"memory"' in clobbers, (source.name, statement)
    assert found == 2
