// sfar_kv_device.cuh -- what the cache's kernels share.
#pragma once
#include <limits.h>

#include "sfar_kv.h"
#include "sfar_prims.cuh"

// Page numbers, slots or lengths that the kernel found out of range.
__device__ __forceinline__ void sfar_kv_fault(SfarCtl *ctl, int at, int where)
{
    sfar_record_code(ctl, SFAR_ERR_INVALID, 0, at, -1, 0, where);
}
