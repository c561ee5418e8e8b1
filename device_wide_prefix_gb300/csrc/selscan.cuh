// Geometry shared by the selective scan's forward and gradient kernels.
#pragma once

#include "sequence.cuh"

namespace dwp {

constexpr int kScanThreads = 128;
constexpr int kNT = 4;          // states of a channel in one thread
constexpr int kScanTile = DWP_SCAN_CHECKPOINT_ROWS;  // rows staged at once, and between saved states

// Code words of the segment map.
constexpr uint32_t kRowHead = 0x80000000u;
constexpr uint32_t kRowTail = 0x40000000u;
constexpr uint32_t kRowSegment = 0x3fffffffu;
constexpr uint32_t kRowOutside = 0xffffffffu;

}  // namespace dwp
