"""Arrays of an MXFP4 call that overlap are refused before a launch (no GPU): by their bytes, not their first
address alone, and rows that interleave in one buffer by their columns."""
import os
import subprocess

import pytest

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

M = 1 << 20
F = 0x7F0000000000  # never dereferenced: every call below fails host validation


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


def refused(a, b, call, *args, **kw):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, stream=0, **kw)
    assert ei.value.status == -1 and "overlaps" in str(ei.value), str(ei.value)
    assert a in str(ei.value) and b in str(ei.value), str(ei.value)


@pytest.mark.parametrize("kind,size", [("bf16", 2), ("f32", 4)])
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("stride", [0, 96])
def test_quantise_and_back(kind, size, tiles, stride):
    r = moe.mx_rows(100, 64, kind, tiles, stride)
    wide, codes, scales = 99 * (stride or 64) * size + 64 * size, 3200, moe.moe_mx_scale_bytes(r)
    up = lambda n: (n - 1) // 16 * 16  # noqa: E731  the last 16-byte place below n
    for inside in (16, up(wide)):
        refused("codes", "x", moe.moe_mx_quantize, r, F, F + inside, F + M)
        refused("scales", "x", moe.moe_mx_quantize, r, F, F + M, F + inside)
        refused("y", "codes", moe.moe_mx_dequantize, r, F + inside, F + M, F)
        refused("y", "scales", moe.moe_mx_dequantize, r, F + M, F + inside, F)
    refused("codes", "x", moe.moe_mx_quantize, r, F + up(codes), F, F + M)
    refused("scales", "x", moe.moe_mx_quantize, r, F + up(scales), F + M, F)
    refused("codes", "scales", moe.moe_mx_quantize, r, F + M, F, F + up(codes))
    refused("codes", "scales", moe.moe_mx_quantize, r, F + M, F + up(scales), F)
    refused("y", "codes", moe.moe_mx_dequantize, r, F, F + M, F + up(codes))
    refused("y", "scales", moe.moe_mx_dequantize, r, F + M, F, F + up(scales))
    rows = moe.mx_rows(100, 64)
    refused("tiles", "scales", moe.moe_mx_tile_scales, rows, F, F + up(200))
    refused("tiles", "scales", moe.moe_mx_tile_scales, rows, F + 512 - 16, F)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_linear(kind):
    T, N, K = 100, 200, 128
    s = moe.mx_shape(T, N, K, kind)
    n = moe.moe_mx_linear_workspace_size(s)
    at = dict(x=F, x_scales=F + M, w=F + 2 * M, w_scales=F + 3 * M, bias=F + 4 * M, residual=F + 5 * M, y=F + 6 * M,
              ws=F + 7 * M)
    if kind == "bf16":
        at["x_scales"] = None
    size = dict(x=T * K * 2 if kind == "bf16" else T * K // 2, x_scales=512, w=N * K // 2, w_scales=1024, bias=4 * N,
                residual=2 * T * N, y=2 * T * N, ws=n)
    for written in ("y", "ws"):
        for other in at:
            if at[other] is None or other == written:
                continue
            a, b = (written, other) if other != "ws" else ("y", "ws")
            for moved in (written, other):
                fixed = other if moved == written else written
                unit = 256 if moved == "ws" else 16
                where = dict(at)  # the moved one starts in the last bytes of the other
                where[moved] = at[fixed] + (size[fixed] - 1) // unit * unit
                refused(a, b, moe.moe_mx_linear, s, *where.values(), ws_bytes=n)


def test_linear_columns_of_one_buffer():
    """x, residual and y as columns of rows of 512 elements: a single shared column is an overlap."""
    T, K, N = 64, 128, 100
    n = moe.moe_mx_linear_workspace_size(moe.mx_shape(T, N, K, "bf16", 512, 512, 512))
    for y, r, a in ((K - 8, 400, "x"), (8, 400, "x"), (512 + 64, 400, "x"), (256, 256 + 96, "residual"),
                    (256, 512 + 160, "residual"), (512 - 96, 128, "x")):
        s = moe.mx_shape(T, N, K, "bf16", 512, 512, 512)
        refused("y", a, moe.moe_mx_linear, s, F, None, F + M, F + 2 * M, None, F + 2 * r, F + 2 * y, F + 3 * M,
                ws_bytes=n)
    # rows of other distances: some row of y meets some row of x
    s = moe.mx_shape(T, N, K, "bf16", 512, 520, 512)
    refused("y", "x", moe.moe_mx_linear, s, F, None, F + M, F + 2 * M, None, None, F + 2 * 160, F + 3 * M, ws_bytes=n)


def test_overlap_of_rows_against_marked_bytes(tmp_path):
    """The check itself, against arrays marked byte by byte: 300,000 drawn pairs, rows apart or not."""
    src = tmp_path / "runs.cpp"
    src.write_text("""
#include "ranges.h"
#include <cstdio>
#include <random>
using moe::Runs;
int main() {
  std::mt19937 g(1);
  auto draw = [&](int lo, int hi) { return lo + (int)(g() % (unsigned)(hi - lo + 1)); };
  int found = 0;
  for (int t = 0; t < 300000; ++t) {
    const int ra = draw(0, 5), rb = draw(0, 5), wa = draw(1, 6), wb = draw(1, 6), sa = wa + draw(0, 9);
    const int sb = draw(0, 1) && sa >= wb ? sa : wb + draw(0, 9), a = draw(1000, 1060), b = draw(1000, 1060);
    bool mark[1300] = {}, meet = false;
    for (int i = 0; i < ra; ++i)
      for (int k = 0; k < wa; ++k) mark[a + i * sa + k] = true;
    for (int i = 0; i < rb; ++i)
      for (int k = 0; k < wb; ++k) meet |= mark[b + i * sb + k];
    const Runs x(reinterpret_cast<void*>((uintptr_t)a), ra, wa, sa), y(reinterpret_cast<void*>((uintptr_t)b), rb, wb, sb);
    if (overlap(x, y) != meet || overlap(y, x) != meet) return 1;
    found += meet;
  }
  std::printf("%d", found);
  // the largest arrays that a call takes
  const int64_t n = 1 << 24, far = (int64_t)1 << 38;
  const Runs big(reinterpret_cast<void*>((uintptr_t)1 << 46), n, 1 << 19, far);
  const Runs next(reinterpret_cast<void*>(((uintptr_t)1 << 46) + (1 << 19)), n, 1 << 19, far);
  return overlap(big, next) || !overlap(big, big) ? 2 : 0;
}
""")
    csrc = os.path.join(os.path.dirname(moe.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc, str(src),
                    "-o", str(tmp_path / "runs")], check=True)
    out = subprocess.run([str(tmp_path / "runs")], capture_output=True, text=True)
    assert out.returncode == 0, out
    assert 30000 < int(out.stdout) < 270000
