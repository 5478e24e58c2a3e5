// int8_f32.hip -- the kernels of int8.h with f32 outputs.
#include "int8.h"

const htk::Int8Launches& htk::int8_f32() { return int8_launches<float>(); }
