// latent.cuh -- the latent cache: host checks shared by its write and read
// paths (latent.cu), its attention (latent_attention.cu) and the page moves
// (pages.cu).
#pragma once

#include "common.cuh"

namespace qvg {

// Host: the shape checks of a cache (the buffers' too, unless `shape_only`).
qvg_status check_latent(const qvg_latent *c, bool shape_only);

}  // namespace qvg
