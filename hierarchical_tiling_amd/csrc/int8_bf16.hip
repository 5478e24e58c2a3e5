// int8_bf16.hip -- the kernels of int8.h with bf16 outputs.
#include "int8.h"

const htk::Int8Launches& htk::int8_bf16() { return int8_launches<u16>(); }
