// ssm_plan_host.cpp -- prints what the state-space block's launch rules
// (csrc/ssm.hpp) choose for sizes given as arguments.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ssm.hpp"

using namespace hyena;

int main(int argc, char** argv) {
  const auto arg = [&](int i) { return i < argc ? std::atoll(argv[i]) : 0; };
  if (argc > 1 && !std::strcmp(argv[1], "scan")) {
    const int64_t B = arg(2), D = arg(3), G = arg(4), N = arg(5), L = arg(6);
    const ScanPlan p = scan_plan(B, D, N, L);
    const ScanBackwardLayout w = scan_backward_layout(B, D, G, N, L);
    const int64_t tile = scan_backward_tile(N, D / G), tiles = (D / G + tile - 1) / tile;
    std::printf("split %d segs %d chunks_per_seg %d waves %d chunks %d splits %d tiles_per %d parts %d\n", p.split, p.segs,
                (int)(p.seg / kScanChunk < w.chunks ? p.seg / kScanChunk : w.chunks), (int)(tile / 4), w.chunks, w.splits,
                (int)((tiles + w.splits - 1) / w.splits), (int)(B * w.chunks));
    return 0;
  }
  if (argc > 1 && !std::strcmp(argv[1], "conv")) {
    const int64_t B = arg(2), D = arg(3), L = arg(4);
    const ConvBackwardGrid g = conv_backward_grid(B, D, L, (int)arg(5) <= 4 ? 4 : (int)arg(5) <= 8 ? 8 : 16);
    std::printf("walks %d\n", (int)(g.seqs / (256 >> g.lper)));
    return 0;
  }
  return 1;
}
