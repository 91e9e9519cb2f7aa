// A rotary plan: the frequency table one set of rotary parameters needs.
#pragma once
#include "internal.cuh"

struct dsa_rope {
  int device;
  int rot_dim;
  int layout;     // dsa_rope_layout
  int max_pos;
  float2* table;  // [max_pos][rot_dim / 2] (cos, sin) of every pair, magnitude included
};
