"""Which kernel takes a product of include/tsenor_ops.h, without a GPU: the library's own rule behind its C
entry points (tests/native/ops_forms.cpp), held to the sizes of tests/ops_sizes.py, so that every kernel has
sizes whose results tests/test_gpu_ops_forms.py compares."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest

import ops_sizes as sizes
import sparse_mask_search_amd as sms
from sparse_mask_search_amd import build

pytestmark = pytest.mark.skipif(shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()),
                                reason="hipcc is not installed")

AT = 0x10000  # an address that nothing reads
P, I, Q = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("forms") / "ops_forms.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.check_call([build.hipcc()] + build._flags() + [
        "-fPIC", "-shared", "-o", so, "-x", "hip", os.path.join(here, "native", "ops_forms.cpp"),
        os.path.join(build.CSRC, "tsenor_ops_abi.cpp")], stderr=subprocess.DEVNULL)
    l = ctypes.CDLL(so)
    l.last_form.restype = ctypes.c_char_p
    l.lds_of_tile.restype = l.workgroups_of_cu.restype = Q
    l.tsenor_grouped_mm.argtypes = [P, Q, Q, P, I, Q, Q, Q, Q, Q, P, P, I, Q, P]
    l.tsenor_grouped_wgrad.argtypes = [P, Q, P, Q, Q, Q, Q, Q, P, P, P, I, Q, Q, P]
    l.tsenor_gemm_int8.argtypes = [P, I, P, Q, Q, P, P, Q, Q, Q, P, P, I, Q, P]
    return l


def form(rule, op, rows, experts, m, k):
    """The form of contiguous operands."""
    if op in ("product", "transposed"):
        t = op == "transposed"
        code = rule.tsenor_grouped_mm(AT, rows, k, AT, int(t), experts, m * k, m if t else k, m, k, AT, AT, 1, m, None)
    elif op == "gradient":
        code = rule.tsenor_grouped_wgrad(AT, m, AT, k, rows, experts, m, k, AT, None, AT, 1, m * k, k, None)
    elif op == "integers":
        code = rule.tsenor_gemm_int8(AT, 3, AT, rows, -(-k // 128) * 128, AT, AT, experts, m, k, AT, AT, 1, m, None)
    else:
        code = rule.tsenor_gemm_int8(AT, 1, None, rows, k, AT, AT, 1, m, k, None, AT, 1, m, None)
    assert code == 0
    return rule.last_form().decode()


def listed():
    for rows, experts, m, k, *forms in sizes.PRODUCTS:
        for op, f in zip(("product", "transposed", "integers"), forms):
            yield op, rows, experts, m, k, f
    for rows, experts, m, k, f in sizes.GRADIENTS:
        yield "gradient", rows, experts, m, k, f


def test_each_size_takes_its_form(rule):
    wrong = [(*case, got) for case in listed() if (got := form(rule, *case[:-1])) != case[-1]]
    assert not wrong, wrong
    assert form(rule, "tokens", 7, 1, 100, 4000) == "tokens"


EVERY = {
    "product": {"few16", "few32", "few64", "few32x32", "any", "staged256x128", *sizes.TILES},
    "transposed": {"any", *sizes.TILES},
    "integers": {"few16", "few32", "few64", "few32x32", *sizes.TILES},
    "gradient": {"any", "64x64", "128x128", "256x256"},
}


@pytest.mark.parametrize("op", sorted(EVERY))
def test_every_form_has_a_size(op):
    cases = [c for c in listed() if c[0] == op]
    assert {c[-1] for c in cases} == EVERY[op]
    for name in sizes.TILES.keys() & EVERY[op]:
        columns, tall, ring, at_once = sizes.TILES[name]
        mine = [c for c in cases if c[-1] == name]
        if op == "gradient":
            ring = 4 if name == "64x64" else ring
            steps = [max(sizes.counts_of(c[1], c[2])) // 32 for c in mine]
            tiles = [-(-c[3] // tall) * -(-c[4] // columns) * c[2] for c in mine]
            assert name == "64x64" or max(tiles) > at_once, "a second tile for a workgroup"
        else:
            steps = [-(-c[4] // 128) * 2 if op == "integers" else 2 * c[4] // 64 for c in mine]
            tiles = [sizes.tiles_of(name, sizes.counts_of(c[1], c[2]), c[3]) for c in mine]
            assert max(t for t, s in zip(tiles, steps) if s > ring + 1) > at_once, "a second tile for a workgroup"
        assert max(steps) > ring + 2, "the loop of whole steps"


@pytest.mark.parametrize("op", ["product", "transposed", "integers"])
def test_half_tiles_in_both_places(op):
    """An expert's last rows, of at most half a tile: behind all whole tiles, and in their places where there are
    four rounds of tiles and more."""
    last = {True: 0, False: 0}
    for c in listed():
        if c[0] == op and c[-1] in sizes.TILES:
            columns, tall, _, at_once = sizes.TILES[c[-1]]
            counts = sizes.counts_of(c[1], c[2])
            across = -(-c[3] // columns)
            groups = min(at_once, across * (c[1] // tall + min(c[2] + 1, c[1])))
            halves = sum(0 < n % tall <= tall // 2 for n in counts)
            last[across * (c[1] // tall) < 4 * groups] += halves if tall > 64 else 0
    assert last[True] > 0 and last[False] > 0, last


def kernels_of_the_library(tmp_path):
    """(name, LDS bytes, vector registers, threads) of every kernel in the library as it was built."""
    readelf = os.path.join(os.path.dirname(os.path.dirname(build.hipcc())), "llvm", "bin", "llvm-readelf")
    if not os.path.exists(readelf):
        pytest.skip("llvm-readelf is not installed")
    data, magic, at, found = open(sms.library_path(), "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", 0, []
    while (at := data.find(magic, at)) >= 0:
        (entries,), entry = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(entries):
            first, size, length = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24:entry + 24 + length] and size:
                obj = tmp_path / "object"
                obj.write_bytes(data[at + first:at + first + size])
                notes = subprocess.check_output([readelf, "--notes", str(obj)], text=True)
                for part in notes.split("  - .agpr_count")[1:]:
                    field = lambda key: re.search(rf"\.{key}:\s+(\S+)", part).group(1)
                    found.append((field("name"), int(field("group_segment_fixed_size")), int(field("vgpr_count")),
                                  int(field("max_flat_workgroup_size"))))
            entry += 24 + length
        at += len(magic)
    return found


def test_workgroups_at_once_fit_a_cu(rule, tmp_path):
    """As many workgroups walk over tiles as a CU holds at one time, by its 160 KB of LDS and its registers (512 a
    lane of each of four SIMDs): more would begin when the first ones have ended."""
    pattern = re.compile(r"product_tile_kernelI.*?KindE(\d)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb(\d)E")
    seen = set()
    for name, lds, registers, threads in kernels_of_the_library(tmp_path):
        if (m := pattern.search(name)) is None or m.group(7) == "0":
            continue
        gradient, columns, rows, _, _, ring = map(int, m.groups()[:6])
        seen.add((gradient, columns, rows, ring))
        assert lds <= rule.lds_of_tile(gradient, columns, rows, ring) + 64 and lds > 64 * (columns + rows) * ring, name
        count = rule.workgroups_of_cu(gradient, columns, rows, ring)
        waves = 4 * (512 // (-(-registers // 8) * 8))
        assert count == min(160 * 1024 // lds, waves // (threads // 64)), (name, lds, registers, count)
    assert seen == {(0, 256, 256, 4), (0, 256, 128, 6), (0, 128, 128, 8), (0, 64, 64, 8), (0, 256, 128, 3),
                    (1, 256, 256, 4), (1, 128, 128, 8)}
