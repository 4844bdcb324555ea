"""Host-side rule of softmax attention's cut tiles (no GPU): a list's blocks, the
blocks of a piece, the pieces of a tile, and the room that the workspace has for
them.  The table kernel's own functions, compiled from its header into a small host
program, on offsets that the library accepts: every piece has blocks, and all cut tiles'
pieces fit their room, also where a list's blocks pass 32 bits.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kimi_delta_attention_bwd_gb300", "csrc")

PROGRAM = r'''
#include <cstdio>
#include <vector>
#include "kda_softmax.cuh"
using namespace kda::smx;
int main() {
  // queries on stdin: "causal tile xb Hq Hkv by_key n, then n + 1 query and n + 1 key offsets"
  // -> tiles, blocks, blocks of a piece, pieces of the cut tiles, their room, pieces without blocks
  int causal, tile, xb, Hq, Hkv, by_key, n;
  while (scanf("%d %d %d %d %d %d %d", &causal, &tile, &xb, &Hq, &Hkv, &by_key, &n) == 7) {
    std::vector<int32_t> cu(n + 1), cuk(n + 1), pre(n + 1);
    for (auto* c : {&cu, &cuk})
      for (auto& v : *c)
        if (scanf("%d", &v) != 1) return 1;
    const auto& own = by_key ? cuk : cu;
    for (int i = 0; i < n; i++) pre[i + 1] = pre[i] + (own[i + 1] - own[i] + tile - 1) / tile;
    const Tiles t{cu.data(), cuk.data(), pre.data(), n, tile, xb, Hq / Hkv, causal, by_key != 0};
    const int H = by_key ? Hkv : Hq, target = kda::SMS;
    const int64_t blocks = t.blocks(0, pre[n], 1), per = piece_blocks(blocks, H, target, xb);
    int64_t pieces = 0, empty = 0, shares = 0;
    for (int s = 0; s < 1024; s++) shares += t.blocks(s, pre[n], 1024);  // (as the kernel's threads take them)
    if (shares != blocks) return 2;
    for (int x = 0; x < pre[n]; x++) {
      const int nb = t.find(x).nb, np = pieces_in(nb, per), len = (nb + np - 1) / np;
      if (np > 1) {
        pieces += np;
        empty += (int64_t)(np - 1) * len >= nb;
      }
    }
    printf("%d %lld %lld %lld %d %lld\n", pre[n], (long long)blocks, (long long)per, (long long)pieces,
           piece_room(target, H), (long long)empty);
  }
  return 0;
}
'''


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("softmax_tiles")
    src, exe = d / "tiles.cu", d / "tiles"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)

    def ask(causal, tile, xb, Hq, Hkv, by_key, lq, lk):
        off = [0, *np.cumsum(lq).tolist(), 0, *np.cumsum(lk).tolist()]
        out = subprocess.run([str(exe)], input=" ".join(map(str, [causal, tile, xb, Hq, Hkv, by_key, len(lq), *off])),
                             check=True, capture_output=True, text=True).stdout.split()
        return [int(x) for x in out]
    return ask


@pytest.mark.parametrize("lq,lk,Hq,Hkv", [([3600000], [77000], 64, 1), ([3600000, 3700000], [38400, 38400], 64, 1),
                                          ([910000], [38000], 1024, 2)])
def test_blocks_past_32_bits(rule, lq, lk, Hq, Hkv):
    """Millions of queries on the keys of few heads: tiles few enough to be cut, and more than 2^31 blocks."""
    tile, xb = 128, 64
    tiles, blocks, per, pieces, room, empty = rule(0, tile, xb, Hq, Hkv, 1, lq, lk)
    assert tiles * Hkv <= 4 * 152 and blocks > 2 ** 31
    assert blocks == sum(-(-a // xb) * (Hq // Hkv) * -(-b // tile) for a, b in zip(lq, lk))
    assert per == -(-blocks * Hkv // 152) and pieces <= room and empty == 0


def test_pieces_fit_their_room(rule):
    r = np.random.RandomState(7)
    for _ in range(60):
        n = int(r.randint(1, 40))
        lq = (2.0 ** r.uniform(0, 15, n)).astype(int).tolist()
        lk = lq if r.rand() < 0.5 else (2.0 ** r.uniform(0, 17, n)).astype(int).tolist()
        Hkv = int(r.choice([1, 2, 4, 8]))
        Hq, by_key, xb = Hkv * int(r.choice([1, 2, 8])), int(r.randint(2)), int(r.choice([32, 64, 128]))
        tile = 128 if by_key else int(r.choice([128, 256]))
        _, _, _, pieces, room, empty = rule(int(r.randint(2)), tile, xb, Hq, Hkv, by_key, lq, lk)
        assert pieces <= room and empty == 0, (lq, lk, Hq, Hkv, by_key, xb, tile)
