#include "attn_common.cuh"
namespace vq3 {
VQ3_BOUNDS_RECORD(attn_wide)
}  // namespace vq3
