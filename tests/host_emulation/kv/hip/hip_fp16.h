// The key-value cache kernels take no types or functions from hip_fp16.h
// (test infrastructure for the bounds-checked CPU runs).
#pragma once
