// fwd_sizes.h -- tiles of the forward kernels whose query tiles meet lists of key blocks.
#pragma once

namespace fa {
namespace {

constexpr int kBM = 128;  // query rows per tile
constexpr int kBN = 128;  // keys per block

}  // namespace
}  // namespace fa
