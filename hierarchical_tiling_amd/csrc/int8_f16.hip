// int8_f16.hip -- the kernels of int8.h with f16 outputs.
#include "int8.h"

const htk::Int8Launches& htk::int8_f16() { return int8_launches<_Float16>(); }
