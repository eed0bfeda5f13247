// See cuda_runtime.h: what the headers name of the driver's types.
#pragma once
struct CUtensorMap { alignas(64) unsigned long long opaque[16]; };
