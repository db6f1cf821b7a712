// qf8_matmul_e4m3_e4m3.hip -- the matrix products of E4M3 rows with E4M3 columns.
#include "qf8_matmul.h"

namespace qf8 {
template int launch_matmul_formats<kE4M3, kE4M3>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);
}
