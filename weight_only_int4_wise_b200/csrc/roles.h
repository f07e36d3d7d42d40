// Which part of a CTA's work a warp of the transposed and wide gated products
// takes (w4a16_dgrad.cu), as plain constant functions of the warp's index. Warps
// 0 (producer) and 1 (MMA issuer) decode nothing, but run through the set-up that
// all warps share: they get block 0 and stage 0, so that what is formed there
// stays inside the parameter arrays.
#pragma once

namespace w4a16 {

constexpr int kFirstDecodeWarp = 2;
constexpr int kGroupWarps = 4;  // warps of a decoding group

// The block (of the CTA's `km`) that the warp's group decodes.
constexpr int block_of_warp(int warp, int km) {
    return warp >= kFirstDecodeWarp ? ((warp - kFirstDecodeWarp) / kGroupWarps) % km : 0;
}

// The first stage that the warp's group decodes; it goes on with every (groups / km)-th.
constexpr int stage_of_warp(int warp, int km) {
    return warp >= kFirstDecodeWarp ? ((warp - kFirstDecodeWarp) / kGroupWarps) / km : 0;
}

}  // namespace w4a16
