"""The walk of the grouped products over their tiles at the largest sizes that the
calls take, on the host: the functions are compiled as they are and every tile they
name has to lie inside its group and the weights, none twice."""
import os
import subprocess

from nvfp4_quantization_precision_gb300 import build as fos_build

SOURCE = r'''
#include <cstdio>
#include <cstring>
#include <vector>
#include "fos_grouped.cuh"
using namespace fos;

// rows per group, weight rows, bytes of a row of codes
static int walk(std::vector<int> rows, int64_t N, int64_t row_bytes, int64_t want_band) {
    const int G = (int)rows.size();
    std::vector<Group> t(G + 1);
    int64_t all = 0;
    t[0] = Group{0, 0};
    for (int g = 0; g < G; ++g) {
        all += rows[g];
        t[g + 1] = Group{(int32_t)all, t[g].tile + (rows[g] + lin::kTokTile - 1) / lin::kTokTile};
    }
    static lin::GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.G = G;
    a.rows = (int)all;
    a.N = (int)N;
    a.tiles_n = (int)((N + lin::kPairM - 1) / lin::kPairM);
    a.band = lin::token_band(all, row_bytes);
    const int64_t tiles = (int64_t)t[G].tile * a.tiles_n;
    auto fail = [&](const char* what, int64_t tile) {
        std::printf("%s: N %lld, rows %lld, %lld bytes a row, band %d, tile %lld of %lld\n", what, (long long)N,
                    (long long)all, (long long)row_bytes, a.band, (long long)tile, (long long)tiles);
        return 1;
    };
    if (want_band && a.band != want_band) return fail("band", 0);
    if (tiles > 0x7FFFFFFF || (int64_t)a.band * a.tiles_n > 0x7FFFFFFF || a.band < 1) return fail("range", 0);
    std::vector<char> seen(tiles <= (1 << 22) ? tiles : 0);
    lin::GroupedTile w;
    w.g = 0;
    const int64_t step = tiles <= (1 << 22) ? 1 : tiles / 100003 + 1;
    for (int64_t i = 0; i < tiles; i = i + step < tiles || i == tiles - 1 ? i + step : tiles - 1) {
        lin::grouped_tile(a, t.data(), (int)i, w);
        if (w.g < 0 || w.g >= G || w.t0 < t[w.g].row || w.t0 >= t[w.g + 1].row || w.live < 1 ||
            w.live > lin::kTokTile || w.t0 + w.live > t[w.g + 1].row || w.n0 < 0 || w.n0 >= N ||
            w.cols < w.live || w.cols > lin::kTokTile)
            return fail("tile", i);
        if (!seen.empty()) {
            const int64_t at = (t[w.g].tile + (w.t0 - t[w.g].row) / lin::kTokTile) * (int64_t)a.tiles_n + w.n0 / lin::kPairM;
            if (seen[at]++) return fail("twice", i);
        }
    }
    return 0;
}

int main() {
    int bad = 0;
    // few tokens, many weight rows of few bytes: 2^28 rows are 2^20 tiles, times 4096 just 2^32
    for (int64_t N : {INT64_C(1) << 28, (INT64_C(1) << 28) + 16, (INT64_C(1) << 28) + (1 << 20), (INT64_C(1) << 29) + 4096,
                      (INT64_C(1) << 30) - 16, (INT64_C(1) << 27), (INT64_C(1) << 24) - 16})
        for (int rows : {1, 192, 193, 1000})
            for (int64_t bytes : {32, 128, 4096}) bad += walk({rows}, N, bytes, 0);
    bad += walk({5, 0, 700}, (INT64_C(1) << 29) - 16, 32, 0);
    // many tokens, few weight rows
    bad += walk({(1 << 30) - 1}, 16, 32, 4882);
    bad += walk({(1 << 30) - 1}, 1024, 128, 0);
    bad += walk({1 << 20, 0, 3, 1 << 20}, 1 << 18, 32, 0);
    // the bands of ordinary sizes: 30 MB of rows, or what there is
    bad += walk({16384}, 2048, 3584, 43);
    bad += walk({8192}, 14336, 4096, 38);
    bad += walk({256}, 2048, 3584, 2);
    bad += walk({1}, 4096, 1 << 20, 1);
    bad += walk({300, 17, 0, 1000}, 1040, 640, 7);
    // more groups than rows
    bad += walk(std::vector<int>(1024, 1), 1 << 20, 32, 0);
    return bad;
}
'''


def test_every_tile_is_inside(tmp_path):
    src, exe = tmp_path / "tiles.cu", tmp_path / "tiles"
    src.write_text(SOURCE)
    r = subprocess.run([fos_build._nvcc(), *fos_build.NVFLAGS, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=dict(os.environ))
    assert r.returncode == 0, r.stdout or r.returncode
