// Generated by gen_gelu_poly.py: least-squares fit of log2 Q(t), Q the upper
// tail of the standard normal, in v = t/3 - 1 for t in [0, 6]; power basis,
// lowest order first; t is clamped at TF_GELU_TCLAMP.  fp16 check over every finite
// input: max 1 ulp, 0.38% of inputs off by one.
#pragma once
#define TF_GELU_TMAX 6.0f
#define TF_GELU_TCLAMP 12.0f
#define TF_GELU_POLY_DEGREE 7
#define TF_GELU_C0 -9.53293514251709f
#define TF_GELU_C1 -14.209549903869629f
#define TF_GELU_C2 -6.033993244171143f
#define TF_GELU_C3 -0.20404955744743347f
#define TF_GELU_C4 0.09173492342233658f
#define TF_GELU_C5 -0.04057419300079346f
#define TF_GELU_C6 0.016779523342847824f
#define TF_GELU_C7 -0.004253455437719822f
// t*Q(t)*sqrt(2 pi)*exp(t^2/2) in 1/t^2, for t in [TF_GELU_TMAX, TF_GELU_TFAR]
#define TF_GELU_TFAR 15.0f
#define TF_GELU_FAR0 0.9999721646308899f
#define TF_GELU_FAR1 -0.9923630952835083f
#define TF_GELU_FAR2 2.4148473739624023f
